"""What lies past a request's last key costs a call nothing, whatever it holds: slots of a block
that nothing was written to, staged entries of absent nodes."""

import pytest
import torch

from tests.test_gpu_attention_forms import DEV, grouped, ints, shared_batch, ver  # noqa: F401
from tests.test_gpu_attention_form_calls import words_of

pytestmark = pytest.mark.gpu


def time_of(call):
    """The fastest of several calls in ms."""
    call(), call()
    best = float("inf")
    for _ in range(7):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        torch.cuda.synchronize()
        a.record()
        call()
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b))
    return best


def caller(ver, x, **kw):
    out, args = torch.empty_like(x.q), (x.q, x.kv, ints(x.table), ints(x.S))
    words, n = words_of(x), ints(x.n)

    def call():
        return ver.tree_attention(*args, layer=1, stage=x.stage, mask=words, n_nodes=n, out=out, **kw)

    return call


def long_batch(fmt, staged, own):
    """Eight requests of one prompt, positions that fill no block, nodes absent from some."""
    return shared_batch(fmt, 64, 8, 2, 16, "binary:2", staged, 30, [own + 5 + b for b in range(8)], [8])


def zeroed(x):
    """The batch's surroundings, NaN in what the tests make, as zeros."""
    for t in (x.kv, x.stage):
        if t is None:
            continue
        if t.dtype == torch.uint8:
            t[(t == 0xFF).all(-1)] = 0
        else:
            torch.nan_to_num_(t, nan=0.0)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("staged", [True, False])
@pytest.mark.parametrize("kw", [{}, dict(softcap=30.0)], ids=["plain", "cap"])
@pytest.mark.parametrize("own", [300, 20000])
def test_unwritten_places_cost_nothing(ver, fmt, staged, kw, own):
    x = long_batch(fmt, staged, own)
    x.n[3] = -1
    call = caller(ver, x, groups=grouped(ver, x), **kw)
    spoiled, took = call().clone(), time_of(call)
    zeroed(x)
    clean, takes = call().clone(), time_of(call)
    assert ver.error() == 0
    live = torch.arange(x.R, device=DEV) <= ints(x.n)[:, None]
    assert torch.equal(spoiled[live], clean[live]) and torch.isfinite(clean).all()
    # clearing them takes a few stores a tile; looking
    # through 300 keys for each output took a hundred times the call
    assert took < 1.5 * takes + 0.02, (took, takes)
