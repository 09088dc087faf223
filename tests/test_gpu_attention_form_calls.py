"""Calls of attention with forms of the scores and shared prefixes that its own tests leave out: strided
queries and outputs, blocks of odd sizes, no mask, wide masks, negative scales and slopes, members without
rows, repeated blocks, long prefixes, thousands of requests, first calls inside a capture.  Bounds
are those derived in test_gpu_attention_forms."""

import numpy as np
import pytest
import torch

from oracle import entries as E
from speculative_decoding_verification_07_gb300 import binding

from tests.test_gpu_attention_forms import DEV, Batch, as_call, forms_of, grouped, ints, poison, random_entries, shared_batch, some_slopes, ver  # noqa: F401

pytestmark = pytest.mark.gpu


def words_of(x):
    return torch.tensor(E.pack(x.bits).view(np.int32), device=DEV)


@pytest.mark.parametrize("fmt,D", [("bf16", 128), ("e4m3", 64), ("fp32", 64)])
@pytest.mark.parametrize("form", [None, "cap", "all"])
def test_strided_queries_and_outputs(ver, fmt, D, form):
    """Queries inside a wider projection, outputs inside a wider buffer whose rest stays as it was."""
    x = shared_batch(fmt, D, 8, 2, 16, "binary:2", True, 9, [40, 2, 33, 140], [3, 1])
    kw = {} if form is None else as_call(forms_of(form, 8))
    g = None if kw.get("window") else grouped(ver, x)
    want = x.run(ver, depth=ints(x.depth), groups=g, **kw)
    wide = torch.full((x.B, x.R, 8 + 4, D), float("nan"), dtype=x.dt, device=DEV)
    wide[:, :, 2:10] = x.q
    x.q = wide[:, :, 2:10]
    room = torch.full((x.B, x.R + 1, 8 + 2, D), 3.0, dtype=x.dt, device=DEV)
    out = x.run(ver, out=room[:, :x.R, 1:9], depth=ints(x.depth), groups=g, **kw)
    assert torch.equal(out, want) and ver.error() == 0
    room[:, :x.R, 1:9] = 3.0
    assert (room == 3.0).all()


@pytest.mark.parametrize("fmt,D", [("bf16", 128), ("bf16", 64), ("e4m3", 128), ("e4m3", 64)])
@pytest.mark.parametrize("BS", [24, 40, 48, 80, 256])
@pytest.mark.parametrize("staged", [False, True])
def test_blocks_of_odd_sizes(ver, fmt, D, BS, staged):
    x = shared_batch(fmt, D, 8, 2, BS, "random:11", staged, 6, [5, 0, 140, 9, 260, 77], [3, 1, 2])
    kw = forms_of("all", 8)
    out = x.run(ver, depth=ints(x.depth), **as_call(kw))
    assert ver.error() == 0
    x.check(out, **kw)
    for kw in ({}, dict(softcap=20.0, slopes=some_slopes(8))):
        out = x.run(ver, depth=ints(x.depth), groups=grouped(ver, x), **as_call(kw))
        assert ver.error() == 0
        x.check(out, **kw)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "fp32"])
@pytest.mark.parametrize("kw", [{}, dict(softcap=20.0), dict(softcap=20.0, slopes=True)], ids=["plain", "cap", "both"])
def test_chains_without_a_mask_and_wide_masks(ver, fmt, kw):
    """No mask is a chain, no counts are all rows; words past a row's bits do not matter."""
    kw = dict(kw, slopes=torch.tensor(some_slopes(4), device=DEV)) if kw.get("slopes") else dict(kw)
    x = shared_batch(fmt, 64, 4, 2, 16, "chain:36", True, 9, [5, 60, 9], [3])
    x.n[:] = 36
    x.bits = np.tile(np.tril(np.ones((37, 37), bool)), (3, 1, 1))
    x.stage[:, :, 1] = x.stage[:1, :, 1].clone()  # (request 1 was drawn with fewer entries)
    words = words_of(x)
    for groups in (None, grouped(ver, x)):
        if groups is None and not kw:
            continue
        call = dict(layer=1, stage=x.stage, groups=groups, **kw)
        want = ver.tree_attention(x.q, x.kv, ints(x.table), ints(x.S), mask=words, n_nodes=ints(x.n), **call)
        assert torch.isfinite(want).all()
        none = ver.tree_attention(x.q, x.kv, ints(x.table), ints(x.S), **call)
        wide = torch.full((3, 37, 5), -1, dtype=torch.int32, device=DEV)
        wide[:, :, :words.shape[2]] = words
        wide[:, :, 1] |= -1 << 5  # bits past the last entry
        more = ver.tree_attention(x.q, x.kv, ints(x.table), ints(x.S), mask=wide, n_nodes=ints(x.n), **call)
        assert torch.equal(none, want) and torch.equal(more, want) and ver.error() == 0


@pytest.mark.parametrize("fmt,D,Hq,H", [("bf16", 128, 4, 2), ("e4m3", 128, 4, 2), ("fp32", 64, 4, 2), ("bf16", 64, 1, 1)])
@pytest.mark.parametrize("scale", [-0.2, 0.0, 0.3])
@pytest.mark.parametrize("sign", [1.0, -1.0, 40.0])
def test_signs_of_scales_and_slopes(ver, fmt, D, Hq, H, scale, sign):
    """Slopes of either sign and steep ones; scores of a negative scale."""
    x = shared_batch(fmt, D, Hq, H, 16, "binary:2", True, 9, [5, 60, 9, 300], [3, 1])
    kw = dict(softcap=10.0, slopes=np.float32(sign) * some_slopes(Hq))
    for groups in (None, grouped(ver, x)):
        out = x.run(ver, depth=ints(x.depth), groups=groups, scale=scale, **as_call(kw))
        assert ver.error() == 0
        x.check(out, scale=scale, **kw)
    kw = dict(slopes=kw["slopes"], window=90)
    out = x.run(ver, depth=ints(x.depth), scale=scale, **as_call(kw))
    assert ver.error() == 0
    x.check(out, scale=scale, **kw)


@pytest.mark.parametrize("fmt,D", [("bf16", 256), ("fp32", 256), ("bf16", 8), ("fp32", 8)])
def test_heads_of_other_sizes(ver, fmt, D):
    x = shared_batch(fmt, D, 4, 2, 16, "binary:2", True, 9, [5, 60, 9, 300], [3, 1])
    kw = forms_of("all", 4)
    out = x.run(ver, depth=ints(x.depth), groups=grouped(ver, x), **as_call(kw))
    assert ver.error() == 0
    x.check(out, **kw)


@pytest.mark.parametrize("fmt,staged", [("bf16", True), ("bf16", False), ("e4m3", True), ("e4m3", False), ("fp32", True)])
@pytest.mark.parametrize("absent", [(0,), (1,), (3,), (0, 1, 2, 3), (0, 2, 4), (4,)])
def test_members_without_rows(ver, fmt, staged, absent):
    """A group's first, last or all requests idle: their rows are zero, the others' as ever."""
    x = shared_batch(fmt, 64, 4, 2, 16, "chain:3", staged, 9, [40, 2, 33, 4, 50], [4, 1])
    g = grouped(ver, x)
    for b in absent:
        x.n[b] = -1
    for kw in ({}, dict(softcap=20.0)):
        out = x.run(ver, groups=g, **kw)
        assert ver.error() == 0
        x.check(out, depth=False, **kw)


def test_no_requests_and_groups_of_one(ver):
    x = shared_batch("bf16", 128, 8, 2, 16, "chain:3", True, 9, [40, 2], [2])
    none = ver.tree_attention(x.q[:0], x.kv, ints(x.table)[:0], ints(x.S)[:0], softcap=3.0, slopes=torch.zeros(8, device=DEV),
                              groups=dict(length=ints([]), members=ints([])))
    assert none.shape == (0, *x.q.shape[1:])
    out = x.run(ver, softcap=3.0, groups=dict(length=ints([144, 0]), members=ints([1, 0])))
    assert ver.error() == 0
    x.check(out, softcap=3.0, depth=False)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "fp32"])
def test_the_same_block_at_several_places(ver, fmt):
    """As copies of it would be, in a prefix, in a request's own blocks, in both."""
    x = shared_batch(fmt, 64, 4, 2, 16, "chain:3", True, 9, [80, 64, 100], [3])
    g = grouped(ver, x)
    copies, again = x.table, x.table.copy()
    for b, to, of in ((0, 4, 1), (0, 11, 2), (1, 10, 9), (2, 12, 0)):
        x.kv[int(copies[b, to])] = x.kv[int(copies[b, of])]
        again[slice(0, 3) if to < 9 else b, to] = copies[b, of]
    for kw in ({}, dict(softcap=20.0, slopes=torch.tensor(some_slopes(4), device=DEV))):
        x.table = copies
        want = x.run(ver, groups=g, **kw)
        x.table = again
        assert torch.equal(x.run(ver, groups=g, **kw), want) and not torch.isnan(want).any()
    assert ver.error() == 0


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_long_prefixes(ver, fmt):
    x = shared_batch(fmt, 64, 4, 1, 64, "chain:2", True, 1200, [70, 5000, 1], [3])  # 76800 positions
    for kw in ({}, dict(softcap=20.0, slopes=some_slopes(4))):
        out = x.run(ver, groups=grouped(ver, x), **as_call(kw))
        assert ver.error() == 0
        x.check(out, depth=False, **kw)
    kw = forms_of("all", 4)
    out = x.run(ver, **as_call(kw))
    assert ver.error() == 0
    x.check(out, depth=False, **kw)


def test_thousands_of_requests(ver):
    """More lots than the list's kernel keeps in shared memory."""
    B = 2100
    x = Batch("bf16", 64, 2, 1, [(7 * b) % 40 for b in range(B)], [b % 4 - 1 for b in range(B)], "chain:2", seed=1)
    rng = np.random.default_rng(0)
    rows = {(b, i) for b in (0, 1, 1023, 1024, 2047, 2048, B - 1, *rng.integers(0, B, 80).tolist()) for i in range(3)}
    for kw in (dict(softcap=3.0), dict(window=9, slopes=some_slopes(2))):
        out = x.run(ver, **as_call(kw))
        assert ver.error() == 0
        x.check(out, depth=False, rows=rows, **kw)


def test_a_first_call_inside_a_capture_and_larger_ones_after_it():
    """The graph's workspace is its own; later calls that need more do not disturb it."""
    small = shared_batch("bf16", 64, 4, 2, 16, "chain:3", True, 9, [40, 2], [2])
    large = shared_batch("bf16", 64, 4, 2, 16, "chain:60", True, 9, [40, 2, 300, 4, 900], [2, 3])
    v = binding.Verifier(0)
    gs, gl = grouped(v, small), grouped(v, large)
    slopes = torch.tensor(some_slopes(4), device=DEV)
    args = [(z.q, z.kv, ints(z.table), ints(z.S)) for z in (small, large)]
    more = [dict(layer=1, stage=z.stage, mask=words_of(z), n_nodes=ints(z.n)) for z in (small, large)]
    other = binding.Verifier(0)
    want = other.tree_attention(*args[0], **more[0], groups=gs, softcap=20.0)
    want_large = other.tree_attention(*args[1], **more[1], slopes=slopes, groups=gl)
    torch.cuda.synchronize()
    graph, out = torch.cuda.CUDAGraph(), torch.zeros_like(small.q)
    with torch.cuda.graph(graph):
        v.tree_attention(*args[0], **more[0], groups=gs, softcap=20.0, out=out)
    for _ in range(3):
        got = v.tree_attention(*args[1], **more[1], slopes=slopes, groups=gl)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(got, want_large)
    assert v.error() == 0 and other.error() == 0
    v.close()
    other.close()


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "fp32"])
@pytest.mark.parametrize("cap,slopes", [(3.0, False), (3.0, True), (5e3, False), (None, True)])
@pytest.mark.parametrize("shared", [False, True])
def test_rows_do_not_depend_on_what_others_see(ver, fmt, cap, slopes, shared):
    """Not even in their last bits: entries that one row sees, other requests' own positions and
    entries, queries of any size beside a row's own."""
    if fmt == "fp32" and shared:
        return
    x = shared_batch(fmt, 64, 8, 2, 16, "chain:6", True, 9, [40, 2, 33, 4], [4])
    x.bits[:] = np.tril(np.ones((7, 7), bool))
    kw = dict(softcap=cap, slopes=torch.tensor(some_slopes(8), device=DEV) if slopes else None, groups=grouped(ver, x) if shared else None)
    clean = x.run(ver, **kw)
    x.check(clean, depth=False, softcap=cap, slopes=some_slopes(8) if slopes else None)
    large = torch.randn(2, 64, generator=torch.Generator(DEV).manual_seed(1), device=DEV) * 300
    for what in (large, torch.full_like(large, float("nan"))):
        if fmt == "e4m3":
            e = poison(fmt, (2, 2), 64)
            if not torch.isnan(what).any():
                e[:] = random_entries((2, 2), fmt, 64, torch.Generator(DEV).manual_seed(2))
                e[..., 64:68] = torch.full((2, 2, 1), 64.0, device=DEV).view(torch.uint8)
        else:
            e = torch.stack([what, what]).to(x.kv.dtype)
        kv, stage, q = x.kv.clone(), x.stage.clone(), x.q.clone()
        p = 9 * 16 + 11
        x.kv[x.table[2, p // 16], 1, :, :, p % 16] = e   # of request 2's own
        x.stage[0, 4, 1] = e                             # seen by the last rows of request 0
        x.q[3, 1] *= 1e3
        out = x.run(ver, **kw)
        assert ver.error() == 0
        assert torch.equal(out[1], clean[1]) and torch.equal(out[0, :4], clean[0, :4])
        keep = [i for i in range(7) if i != 1]
        assert torch.equal(out[3, keep], clean[3, keep])
        assert not torch.equal(out[2], clean[2]) and not torch.equal(out[0, 4:], clean[0, 4:]) and not torch.equal(out[3, 1], clean[3, 1])
        x.kv, x.stage, x.q = kv, stage, q


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("staged", [False, True])
@pytest.mark.parametrize("tree", ["random:25", "chain:150"])
def test_rows_that_see_one_key_give_its_value_back(ver, fmt, staged, tree):
    """Exactly: codes of 4 significant bits times a power of two, or bf16 values."""
    n = int(tree.split(":")[1])
    x = Batch(fmt, 128, 8, 2, [333, 0, 341], [n, n // 2, n], tree, staged=staged, seed=4, size=2.0)
    out = x.run(ver, depth=ints(x.depth), window=1, softcap=67.2, slopes=torch.tensor(some_slopes(8), device=DEV))
    assert ver.error() == 0
    for b in range(3):
        for h in range(8):
            want = torch.tensor(x.V[b][x.S[b]:x.S[b] + x.n[b] + 1, h // 4], device=DEV)
            assert torch.equal(out[b, :x.n[b] + 1, h].double(), want)


def test_outputs_of_groups_that_overlap_are_refused(ver):
    table, S = ints([[1, 2], [1, 2]]), ints([32, 32])
    both = ints([0, 0, 0])
    for length, members in ((both[:2], both[:2]), (both[:2], both[1:]), (S, both[:2]), (both[:2], S), (table.view(-1)[1:3], both[:2])):
        with pytest.raises((ValueError, binding.SvError)):
            ver.prefix_groups(table, S, 16, out=dict(length=length, members=members))
    assert ver.error() == 0 and S.tolist() == [32, 32]
