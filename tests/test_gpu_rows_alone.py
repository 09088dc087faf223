"""A row's result does not depend, in its last bit either, on the rows beside it: over many draws, with
scores that rise above a row's first reference by less than what moves it while its neighbours'
move.  Values are rows of a unit matrix, so that outputs are sums of few weights and show their bits."""

import pytest
import torch

from tests.test_gpu_attention_forms import DEV, Batch, grouped, shared_batch, some_slopes, ver  # noqa: F401

pytestmark = pytest.mark.gpu


def show_weights(x):
    """Position p's values become row p % D of a unit matrix."""
    D = x.D
    for b in range(x.B):
        p = torch.arange(int(x.S[b]), device=DEV)
        v = torch.nn.functional.one_hot(p % D, D)[:, None].expand(-1, x.H, -1)
        at = (torch.tensor(x.table[b], device=DEV).long()[p // x.BS], 1, 1, slice(None), p % x.BS)
        if x.fmt != "e4m3":
            x.kv[at] = v.to(x.kv.dtype)
            continue
        codes = torch.zeros(*v.shape[:2], x.kv.shape[-1], dtype=torch.uint8, device=DEV)
        codes[..., :D] = v * 0x38  # 1
        codes[..., D:D + 4] = torch.ones(1, device=DEV).view(torch.uint8)
        x.kv[at] = codes


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "fp32"])
@pytest.mark.parametrize("kw", [dict(window=10 ** 6), dict(softcap=30.0), dict(slopes=True)], ids=["window", "cap", "slopes"])
@pytest.mark.parametrize("S,B", [(119, 96), (2900, 4)])
def test_queries_of_any_size_beside_a_row(ver, fmt, kw, S, B):
    """72 rows a head, so that a warp's lanes are rows of nine entries and it weighs all keys of a tile."""
    kw = dict(kw, slopes=torch.tensor(some_slopes(16) * 0.01, device=DEV)) if kw.get("slopes") else kw
    for seed in range(3):
        x = Batch(fmt, 128, 16, 2, [S] * B, [8] * B, "chain:8", seed=seed, size=1.5)
        show_weights(x)
        x.stage[:, :, 1, 1] = 0
        clean = x.run(ver, **kw)
        for size in (3.0, 10.0, 60.0):
            keep = x.q.clone()
            x.q[:, [1, 4]] *= size
            out = x.run(ver, **kw)
            x.q.copy_(keep)
            others = [0, 2, 3, 5, 6, 7, 8]
            assert torch.equal(out[:, others], clean[:, others]), (seed, size)
            assert not torch.equal(out[:, [1, 4]], clean[:, [1, 4]])
    assert ver.error() == 0


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("kw", [{}, dict(softcap=30.0)], ids=["plain", "cap"])
def test_queries_of_other_requests(ver, fmt, kw):
    """Rows of all requests of a group lie in one item, side by side in a warp."""
    for seed in range(4):
        x = shared_batch(fmt, 64, 8, 2, 16, "chain:1", True, 200, [300, 20 + seed, 33, 1500], [4], size=1.5)
        show_weights(x)
        g = grouped(ver, x)
        clean = x.run(ver, groups=g, **kw)
        for size in (3.0, 10.0, 60.0):
            keep = x.q.clone()
            x.q[1] *= size
            out = x.run(ver, groups=g, **kw)
            x.q.copy_(keep)
            assert torch.equal(out[[0, 2, 3]], clean[[0, 2, 3]]), (seed, size)
    assert ver.error() == 0
