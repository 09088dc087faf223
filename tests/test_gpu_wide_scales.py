"""Attention over 8-bit caches whose entries' V scales differ widely: all-zero V
rows that a row weighs most, V that is tiny in the first tiles, scales spread
over all exponents; against the fp64 definition on what the cache holds.

Bounds, derived before any run.  Weights have 9 significant bits where they are
within 2^-18 of a row's largest product of weight and V scale: 2^-9, within the
2^-8 below; fp32 terms below 2^-10; both in units of sum p |v|.  Smaller ones
lose at most 3 x 2^-26 < 2^-24 of that largest product (taken as 2^-115 at
least) for each unit of a code, and the scale of a row that is not all zeros is
at most max|v| / 224.  The output's own rounding is 2^-8 |o|.
"""

import os

import numpy as np
import pytest
import torch

from oracle import entries as E
from speculative_decoding_verification_07_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BS = 16


@pytest.fixture(scope="module")
def ver():
    if not os.path.exists(binding.LIB_PATH):
        from speculative_decoding_verification_07_gb300 import build
        build.build()
    v = binding.Verifier(0)
    yield v
    v.close()


def ints(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)


def check(ver, q, k, v, cache=None):
    """q [G, D], k, v [n, D] fp64: one KV head, all keys seen by one entry's G heads."""
    (G, D), n = q.shape, k.shape[0]
    blocks = -(-n // BS)
    kv = torch.zeros(blocks, 1, 2, 1, BS, D + E.TAIL, dtype=torch.uint8, device=DEV)
    table = torch.randperm(blocks, generator=torch.Generator().manual_seed(n)).int()[None].to(DEV)
    bf = lambda x: torch.tensor(x, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    keep = np.arange(n) if cache is None else np.flatnonzero(cache)  # entries that are written at all
    for first in range(0, n, 64):  # entries that are not written stay zero-filled
        at = keep[(keep >= first) & (keep < first + 64)]
        for run in np.split(at, np.flatnonzero(np.diff(at) > 1) + 1):
            if run.size:
                ver.kv_append(bf(k[run])[None, :, None], bf(v[run])[None, :, None], ints([run[0]]), kv=kv, block_table=table)
    zero = ints([0])
    held = ver.kv_read(torch.empty(1, n, 2, 1, D, device=DEV), zero, kv=kv, block_table=table)[0, :, :, 0].double().cpu().numpy()
    got = ver.tree_attention(bf(q)[None, None], kv, table, ints([n - 1]))[0, 0].double().cpu().numpy()
    assert ver.error() == 0
    rows = kv[table[0].long(), 0, 1, 0].reshape(-1, D + E.TAIL)[:n].cpu().numpy()
    codes = np.abs(E.e4m3_value(rows[:, :D]))
    qd = bf(q).double().cpu().numpy()
    assert np.isfinite(held).all()
    for g in range(G):
        o, size, scores = E.attend(qd[g], held[:, 0], held[:, 1], np.ones(n, bool), D ** -0.5)
        assert scores < 64
        s = held[:, 0] @ qd[g] * D ** -0.5
        p = np.exp(s - s.max())
        p /= p.sum()
        floor = 2.0 ** -24 * max((p * np.abs(held[:, 1]).max(-1)).max() / 224, 2.0 ** -115) * codes.sum(0)
        tol = (2.0 ** -8 + 2.0 ** -10) * size + 2.0 ** -8 * np.abs(o) + floor
        d = np.abs(got[g] - o)
        assert (d <= tol).all(), (g, d.max(), (d / tol).max())


def keys(rng, n, D, lead):
    """Directions, queries and keys: keys of lead l score l nats, the others little."""
    u = rng.choice([-1.0, 1.0], D)
    return u, lead[:, None] * u / D ** 0.5 + 0.05 * rng.standard_normal((n, D))


# rows a head: 4 (the tile holds them four times), 40 (twice), 100, 150 (two row tiles)
@pytest.mark.parametrize("G,D", [(4, 128), (40, 128), (100, 64), (150, 128)])
@pytest.mark.parametrize("n", [8, 64, 1000])
@pytest.mark.parametrize("lead", [4.0, 8.0, 10.0, 12.0, 14.0])
def test_zero_rows_that_weigh_most(ver, G, D, n, lead):
    rng = np.random.default_rng(int(n + lead))
    for std in (2.0 ** -14, 0.05, 1.0, 2.0 ** 10):
        leads = np.zeros(n)
        leads[[0, n // 2]] = lead
        u, k = keys(rng, n, D, leads)
        v = std * rng.standard_normal((n, D))
        v[[0, n // 2]] = 0
        q = np.repeat(u[None], G, 0) * rng.choice([1.0, 0.5, 0.75], (G, 1))
        check(ver, q, k, v)


@pytest.mark.parametrize("G,D", [(4, 128), (40, 64), (150, 128)])
@pytest.mark.parametrize("course", ["tiny first", "tiny last", "all tiny", "spread", "rising", "huge first", "one channel"])
def test_scales_of_all_sizes(ver, G, D, course):
    rng = np.random.default_rng(len(course) + G)
    n = 700
    e = {"tiny first": np.where(np.arange(n) < 300, -118, 0), "tiny last": np.where(np.arange(n) < 300, 0, -118),
         "all tiny": np.full(n, -100), "spread": rng.integers(-118, 20, n), "rising": np.arange(n) // 5 - 118,
         "huge first": np.where(np.arange(n) < 40, 90, -20), "one channel": np.zeros(n, int)}[course]
    u, k = keys(rng, n, D, 4 * rng.random(n) * (rng.random(n) < 0.1))
    v = rng.standard_normal((n, D)) * 2.0 ** e[:, None]
    if course == "one channel":
        v[rng.random(n) < 0.01, 3] = 1000.0
    check(ver, np.repeat(u[None], G, 0) * rng.choice([1.0, -0.5], (G, 1)), k, v)


@pytest.mark.parametrize("G", [1, 4, 31, 40, 100, 150, 250])
@pytest.mark.parametrize("n", [50, 90, 700])
def test_steep_scores_beside_rows_that_see_nothing(ver, G, n):
    """Heads that fill no whole warp: the others' references move all the same."""
    rng = np.random.default_rng(G + n)
    q, k = 3 * rng.standard_normal((G, 128)), rng.standard_normal((n, 128))
    check(ver, q, k * np.where(np.arange(n) % 40 > 35, 1.5, 0.5)[:, None], rng.standard_normal((n, 128)))


@pytest.mark.parametrize("G", [4, 40, 150])
@pytest.mark.parametrize("n", [20, 500])
def test_zero_filled_entries(ver, G, n):
    """Entries that nothing was written to are zeros, scale included."""
    rng = np.random.default_rng(n)
    u, k = keys(rng, n, 128, np.zeros(n))
    written = np.arange(n) >= n - 15
    k[~written] = 0
    check(ver, np.repeat(u[None], G, 0), k, rng.standard_normal((n, 128)), written)


@pytest.mark.parametrize("staged", [True, False])
def test_scales_of_zero_rows(ver, staged):
    """1 for a key, the smallest for a value, in whatever head and entry."""
    g = torch.Generator(DEV).manual_seed(4)
    k, v = torch.randn(2, 1, 20, 3, 64, generator=g, device=DEV).bfloat16()
    k[0, 3, 1], v[0, 3, 2], v[0, 17] = 0, 0, 0
    place = dict(stage=torch.zeros(1, 20, 1, 2, 3, 64 + E.TAIL, dtype=torch.uint8, device=DEV)) if staged else \
        dict(kv=torch.zeros(2, 1, 2, 3, BS, 64 + E.TAIL, dtype=torch.uint8, device=DEV), block_table=ints([[1, 0]]))
    ver.kv_append(k, v, ints([0]), **place)
    assert ver.error() == 0
    rows = place["stage"][0, :, 0] if staged else place["kv"][[1, 0], 0].permute(0, 3, 1, 2, 4).flatten(0, 1)[:20]
    scale = rows[..., 64:68].contiguous().view(torch.float32)[..., 0].cpu()
    assert scale[3, 0, 1] == 1 and scale[3, 1, 2] == 2.0 ** -126 and (scale[17, 1] == 2.0 ** -126).all()
    others = torch.ones_like(scale, dtype=torch.bool)
    others[3, 0, 1] = others[3, 1, 2] = others[17, 1] = False
    assert (scale[others] > 2.0 ** -10).all() and (scale[others] < 1).all()
    assert not rows[17, 1, :, :64].any()
