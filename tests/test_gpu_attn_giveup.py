"""Waits of the attention kernels that give up (a limit of a few polls): the error
is raised, nothing is written that would depend on them, and the next call on the
same workspace is right."""
import pytest
import torch

import gated_deltanet_speculative_gb300 as gdn

from test_gpu_attn import TYPES, Round

pytestmark = pytest.mark.gpu
TIMEOUT = 32


@pytest.fixture(autouse=True)
def usual_limit():
    yield
    gdn.debug_attn_wait_limit()


# (tokens, rows): items that lie whole in a run, and items that runs share
SHAPES = {"steps": ([700, 90, 3, 1500] * 60, [1] * 240), "one step": ([30000], [1]),
          "windows": ([300, 20, 129] * 70, [16, 3, 7] * 70), "one window": ([20000], [16]), "tree": ([5000, 300], [16, 9])}


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("act,kv", TYPES)
def test_waits_that_give_up_at_once_write_nothing(act, kv, d, shape):
    lengths, rows = SHAPES[shape]
    r = Round(lengths, rows, d=d, act=act, kv=kv, hq=8, hkv=2, page=64, step="step" in shape, tree=shape == "tree")
    want = r.run()
    size = gdn.attn_workspace_size(r.dims, r.pool.dev(), r.pool.S, r.q.shape[0])
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
    gdn.debug_attn_wait_limit(0)
    out = r.run(check_error=TIMEOUT, workspace=ws)
    assert (out == -77.0).all()
    gdn.debug_attn_wait_limit()
    assert torch.equal(r.run(workspace=ws), want)


class Either:
    def __eq__(self, bits):
        return bits in (0, TIMEOUT)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("act,kv", TYPES[::3])
def test_what_is_written_is_right_wherever_a_wait_gives_up(act, kv, shape):
    """Some waits end and some do not; the workspace holds another call's pieces."""
    lengths, rows = SHAPES[shape]
    r = Round(lengths, rows, d=128, act=act, kv=kv, hq=8, hkv=2, page=64, step="step" in shape, tree=shape == "tree")
    want = r.run()
    size = gdn.attn_workspace_size(r.dims, r.pool.dev(), r.pool.S, r.q.shape[0])
    ws = torch.empty((size,), dtype=torch.uint8, device="cuda")
    q, other = r.q, torch.randn(r.q.shape, generator=torch.Generator().manual_seed(9)).to(act)
    for polls in (1, 2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64, 100, 200, 500, 2000):
        r.q = other
        r.run(workspace=ws)
        r.q = q
        gdn.debug_attn_wait_limit(polls)
        out = r.run(check_error=Either(), workspace=ws)
        gdn.debug_attn_wait_limit()
        written = out != -77.0
        assert torch.equal(out[written], want[written]), f"{polls} polls"
        assert torch.equal(r.run(workspace=ws), want), f"after {polls} polls"
