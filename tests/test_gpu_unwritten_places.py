"""What lies past a request's last key costs a call nothing, whatever it holds: slots of a block
that nothing was written to, staged entries of absent nodes.  Values that rows do see cost the
look-up of those values, not of every key."""

import pytest
import torch

from tests.test_gpu_attention_forms import DEV, Batch, grouped, ints, poison, shared_batch, ver  # noqa: F401
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
    assert took < 4 * takes + 0.1, (took, takes)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("kw", [{}, dict(softcap=30.0)], ids=["plain", "cap"])
def test_a_value_that_rows_see(ver, fmt, kw):
    """One NaN among 20000 own positions of one request: its rows are NaN in that column, all others'
    as before; one in an entry: the rows that see it."""
    x = long_batch(fmt, True, 20000)
    zeroed(x)
    call = caller(ver, x, groups=grouped(ver, x), **kw)
    clean, takes = call().clone(), time_of(call)
    p, col = 30 * 16 + 12345, 11
    bad = 0x7F if fmt == "e4m3" else float("nan")
    x.kv[x.table[2, p // 16], 1, 1, :, p % 16, col] = bad
    x.stage[4, 1, 1, 1, :, col] = bad
    out, took = call().clone(), time_of(call)
    assert ver.error() == 0
    want = clean.clone()
    want[2, :x.n[2] + 1, :, col] = float("nan")
    sees = torch.tensor(x.bits[4, :, 1], device=DEV) & (torch.arange(x.R, device=DEV) <= int(x.n[4]))
    want[4, sees, :, col] = float("nan")
    assert sees.any() and torch.equal(torch.isnan(out), torch.isnan(want))
    keep = ~torch.isnan(want)
    assert torch.equal(out[keep], want[keep])
    assert took < 4 * takes + 0.2, (took, takes)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("staged", [True, False])
def test_values_in_more_tiles_than_are_noted(ver, fmt, staged):
    """Infinities all over the own positions of two requests, of either sign and both."""
    x = shared_batch(fmt, 128, 8, 2, 16, "chain:2", staged, 9, [3000, 40, 2900, 7], [4])
    g = grouped(ver, x)
    zeroed(x)
    clean = x.run(ver, groups=g)
    want = clean.clone()
    inf = (lambda s: s * float("inf")) if fmt == "bf16" else (lambda s: 0x7F)  # (8-bit values have NaN alone)
    for b, cols in ((0, {3: 1, 70: -1}), (2, {5: -1})):
        t = torch.tensor(x.table[b], device=DEV).long()
        for p in range(9 * 16, int(x.S[b]), 61):
            for c, s in cols.items():
                x.kv[t[p // 16], 1, 1, :, p % 16, c] = inf(s)
        for c, s in cols.items():
            want[b, :x.n[b] + 1, :, c] = s * float("inf") if fmt == "bf16" else float("nan")
    if fmt == "bf16":  # one of the other sign in the last own position: NaN
        p = int(x.S[0]) - 1
        x.kv[x.table[0, p // 16], 1, 1, :, p % 16, 3] = -float("inf")
        want[0, :x.n[0] + 1, :, 3] = float("nan")
    out = x.run(ver, groups=g)
    assert ver.error() == 0
    assert torch.equal(torch.isnan(out), torch.isnan(want)) and torch.equal(out.nan_to_num(), want.nan_to_num())


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("window", [600, 40])
def test_values_at_a_windows_edge(ver, fmt, window):
    """Positions that rows near the root see and deeper ones do not, in requests of their own."""
    x = Batch(fmt, 64, 4, 2, [2000, 130], [30, 30], "chain:30", seed=3, trees=[0, 0])
    call = caller(ver, x, depth=ints(x.depth), window=window)
    zeroed(x)
    clean = call().clone()
    for b, S in ((0, 2000), (1, 130)):
        if S < window:
            continue
        for d in (0, 7, 20):  # the row at depth d is the last that sees the position
            p = S + d - window + 1
            x.kv[x.table[b, p // 16], 1, :, :, p % 16] = poison(fmt, (2, 2), 64)
        seen = torch.arange(31, device=DEV) <= 20
        out = call()
        assert ver.error() == 0
        assert torch.isnan(out[b, seen]).all() and torch.equal(out[b, ~seen], clean[b, ~seen])
