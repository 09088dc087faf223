"""Captured calls with forms and groups, replayed after the lengths, tables, counts, masks and groups that
they read have changed in place: the list of items is made anew by every replay."""

import numpy as np
import pytest
import torch

from tests.test_gpu_attention_form_calls import words_of
from tests.test_gpu_attention_forms import DEV, Batch, as_call, forms_of, ints, shared_batch, some_slopes, ver  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("form", ["none", "cap", "slopes", "window"])
def test_replays_read_what_is_there(ver, fmt, form):
    kw = {} if form == "none" else forms_of(form, 8)
    x = shared_batch(fmt, 64, 8, 2, 16, "binary:2", True, 20, [5, 300, 33, 90, 2, 700], [4, 2])
    table, S, n, words, depth = ints(x.table), ints(x.S), ints(x.n), words_of(x), ints(x.depth)
    out, call = torch.zeros_like(x.q), as_call(kw)  # (what the graph reads outlives it)

    def step():
        groups = ver.prefix_groups(table, S, 16, least=1)
        return ver.tree_attention(x.q, x.kv, table, S, layer=1, stage=x.stage, mask=words, n_nodes=n, depth=depth, groups=groups, out=out, **call)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    rng = np.random.default_rng(3)
    for turn in range(4):
        if turn:
            # other lengths, and one request whose prefix becomes its own
            S.copy_(ints([20 * 16 + int(v) for v in rng.integers(0, 5, 6)] if turn == 1 else rng.integers(0, np.asarray(x.S) + 1)))
            n.copy_(ints(rng.integers(-1, x.R, 6)))
            if turn == 2:
                table[2, 3] = int(table[1, 21])
            x.q.mul_(1.1)
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        out.fill_(7.0)
        assert torch.equal(step(), got) and not torch.isnan(got).any()
    assert ver.error() == 0


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_replays_of_prompts(ver, fmt):
    """Row blocks' ranges too."""
    x = Batch(fmt, 128, 8, 2, [400, 0, 130], [299, 200, 131], "chain:299", seed=7)
    S, n, table, words = ints(x.S), ints(x.n), ints(x.table), words_of(x)
    slopes = torch.tensor(some_slopes(8), device=DEV)
    call = dict(layer=1, stage=x.stage, mask=words, n_nodes=n, window=150, slopes=slopes)
    out = torch.zeros_like(x.q)
    ver.tree_attention(x.q, x.kv, table, S, out=out, **call)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ver.tree_attention(x.q, x.kv, table, S, out=out, **call)
    for lens, counts in (([400, 0, 130], [299, 200, 131]), ([3, 0, 128], [0, -1, 40]), ([399, 0, 0], [150, 299, 299])):
        S.copy_(ints(lens)), n.copy_(ints(counts))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(ver.tree_attention(x.q, x.kv, table, S, **call), got)
    assert ver.error() == 0
