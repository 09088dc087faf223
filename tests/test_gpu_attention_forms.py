"""sv_tree_attention with capped scores, distance biases, windows and shared prefixes, and
sv_prefix_groups, against the fp64 definitions.

Bounds, derived before any run (u = 2^-24), in units of sum p |v|, n keys seen:
  scores        the product's (D + 3) u times the largest sum |q||k| scale; the cap's slope is at
                most 1, and its own steps (a division, the tanh, a product, powers of two) add 8 u
                of the score; a distance term two roundings of its size
  fp32          twice the scores' error (a weight and the normaliser), and the sums, (n + 16) u each
  bf16          twice the scores' error, weights rounded to 8 bits 2^-8, the sums below 2^-10, and
                the output's 2^-8 |o|
"""

import os

import numpy as np
import pytest
import torch

from oracle import entries as E
from speculative_decoding_verification_07_gb300 import binding
from speculative_decoding_verification_07_gb300 import workloads as W

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
TORCH = {"bf16": torch.bfloat16, "fp32": torch.float32, "e4m3": torch.uint8}


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


def f64(t):
    return t.detach().cpu().numpy() if t.dtype == torch.uint8 else t.detach().double().cpu().numpy()


def random_entries(shape, fmt, D, g, size=1.0):
    x = torch.randn(*shape, D, generator=g, device=DEV) * size
    if fmt != "e4m3":
        return x.to(TORCH[fmt])
    out = torch.zeros(*shape, D + E.TAIL, dtype=torch.uint8, device=DEV)
    e = torch.randint(-9, -5, tuple(shape), generator=g, device=DEV).float()
    out[..., :D] = (x * 80).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    out[..., D:D + 4] = torch.exp2(e).unsqueeze(-1).view(torch.uint8)
    return out


def poison(fmt, shape, D):
    if fmt == "e4m3":
        return torch.full((*shape, D + E.TAIL), 0xFF, dtype=torch.uint8, device=DEV)
    return torch.full((*shape, D), float("nan"), dtype=TORCH[fmt], device=DEV)


class Batch:
    """Random inputs in poisoned surroundings, some requests' leading blocks shared with
    their left neighbours' (common[b] of them)."""

    def __init__(self, fmt, D, Hq, H, S, n, tree, *, staged=True, BS=16, seed=0, common=None, size=1.0, trees=None):
        rng = np.random.default_rng(seed)
        g = torch.Generator(DEV).manual_seed(seed)
        self.fmt, self.D, self.Hq, self.H, self.BS, self.staged = fmt, D, Hq, H, BS, staged
        self.S, self.n, B, L = np.asarray(S), np.asarray(n), len(S), 2
        par = [W.tree_shape(tree, np.random.default_rng(x)) for x in (trees or [0] * B)]
        R = len(par[0]) + 1
        self.B, self.R = B, R
        both = [E.ancestors(p, int(m)) for p, m in zip(par, self.n)]
        self.bits = np.stack([x[0] for x in both])
        self.depth = np.stack([x[1] for x in both])
        have = self.S + (0 if staged else np.maximum(self.n + 1, 0))
        blocks = -(-have // BS)
        common = np.zeros(B, int) if common is None else np.asarray(common)
        order = rng.permutation(int(blocks.sum()) + 3)
        self.table = np.full((B, max(1, blocks.max())), -1, np.int32)
        at = 0
        for b in range(B):
            c = common[b]
            self.table[b, :c] = self.table[b - 1, :c]
            self.table[b, c:blocks[b]] = order[at:at + blocks[b] - c]
            at += blocks[b] - c
        self.kv = poison(fmt, (len(order), L, 2, H, BS), D)
        self.stage = poison(fmt, (B, R, L, 2, H), D) if staged else None
        self.K, self.V = [], []
        for b in range(B):
            t = torch.tensor(self.table[b], device=DEV).long()
            p = torch.arange(have[b], device=DEV)
            new = p >= common[b] * BS
            if have[b]:
                e = random_entries((have[b], 2, H), fmt, D, g, size)
                self.kv[t[p[new] // BS], 1, :, :, p[new] % BS] = e[new]
            e = self.kv[t[p // BS], 1, :, :, p % BS]
            if staged and self.n[b] >= 0:
                s = random_entries((self.n[b] + 1, 2, H), fmt, D, g, size)
                self.stage[b, :self.n[b] + 1, 1] = s
                e = torch.cat([e, s])
            v = E.decode(f64(e), fmt, D)
            self.K.append(v[:, 0]), self.V.append(v[:, 1])
        self.dt = torch.float32 if fmt == "fp32" else torch.bfloat16
        self.q = torch.randn(B, R, Hq, D, generator=g, device=DEV).to(self.dt)

    def run(self, ver, out=None, **kw):
        out = torch.full_like(self.q, 3.0) if out is None else out
        words = torch.tensor(E.pack(self.bits).view(np.int32), device=DEV)
        ver.tree_attention(self.q, self.kv, ints(self.table), ints(self.S), layer=1, stage=self.stage, mask=words,
                           n_nodes=ints(self.n), out=out, **kw)
        return out

    def check(self, out, softcap=None, slopes=None, window=None, scale=None, depth=True, rows=None):
        got, qd, sc = f64(out), f64(self.q), self.D ** -0.5 if scale is None else scale
        G = self.Hq // self.H
        for b in range(self.B):
            for i in range(self.R):
                if i > self.n[b]:
                    assert not got[b, i].any()
                    continue
                if rows is not None and (b, i) not in rows:
                    continue
                m, S = self.n[b] + 1, self.S[b]
                d = self.depth[b] if depth else np.arange(self.R)
                seen = np.concatenate([np.ones(S, bool), self.bits[b, i, :m]])
                far = np.abs(d[i] - np.concatenate([np.arange(-S, 0), d[:m]]))
                for h in range(self.Hq):
                    o, size_v, size_s, size_d = E.attend_shaped(
                        qd[b, i, h], self.K[b][:, h // G], self.V[b][:, h // G], seen, sc, far, softcap,
                        None if slopes is None else float(slopes[h]), window)
                    scores = 2 * ((self.D + 11) * U * size_s + 2 * U * size_d)
                    if self.fmt == "fp32":
                        tol = (scores + 2 * (seen.sum() + 16) * U) * size_v
                    else:
                        tol = (2.0 ** -8 + 2.0 ** -10 + scores) * size_v + 2.0 ** -8 * np.abs(o)
                    bad = np.abs(got[b, i, h] - o) > tol
                    assert not bad.any(), (b, i, h, np.flatnonzero(bad)[:4], got[b, i, h][bad][:4], o[bad][:4])


def some_slopes(Hq):
    return np.float32(2.0) ** (-8 * np.arange(1, Hq + 1, dtype=np.float32) / Hq)


FORMS = {"cap": dict(softcap=3.0), "slopes": dict(slopes=True), "window": dict(window=40),
         "all": dict(softcap=20.0, slopes=True, window=130), "window1": dict(window=1)}
SHAPES = [  # fmt, D, Hq, H, BS
    ("bf16", 128, 8, 2, 16), ("e4m3", 128, 8, 2, 16), ("fp32", 64, 4, 4, 16), ("bf16", 64, 7, 1, 8), ("e4m3", 64, 6, 2, 32),
    ("bf16", 80, 6, 3, 24), ("e4m3", 96, 4, 2, 16), ("fp32", 128, 4, 1, 1), ("bf16", 128, 16, 1, 64)]


def forms_of(name, Hq):
    kw = dict(FORMS[name])
    if kw.get("slopes"):
        kw["slopes"] = some_slopes(Hq)
    return kw


def as_call(kw):
    return {k: torch.tensor(v, device=DEV) if k == "slopes" else v for k, v in kw.items()}


@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("fmt,D,Hq,H,BS", SHAPES)
def test_forms(ver, fmt, D, Hq, H, BS, form):
    kw = forms_of(form, Hq)
    for staged, tree, S, n in ((True, "random:9", [0, 1, 31, 200, 517], [9, 0, -1, 5, 9]),
                               (False, "binary:3", [0, 127, 128, 129, 300], [14, 14, 3, 0, 14])):
        x = Batch(fmt, D, Hq, H, S, n, tree, staged=staged, BS=BS, seed=D + len(form), size=2.0, trees=range(5))
        out = x.run(ver, depth=ints(x.depth), **as_call(kw))
        assert ver.error() == 0
        x.check(out, **kw)
        assert torch.equal(out, x.run(ver, depth=ints(x.depth), **as_call(kw)))


@pytest.mark.parametrize("fmt,Hq,H", [("bf16", 8, 1), ("e4m3", 28, 4), ("bf16", 4, 4), ("fp32", 4, 2)])
@pytest.mark.parametrize("form", ["cap", "slopes", "window", "all"])
@pytest.mark.parametrize("staged", [False, True])
def test_forms_of_prompts(ver, fmt, Hq, H, form, staged):
    """Chains of many row blocks and of several tiles of entries, with no depth and with a chain's
    given; a last block of few rows, a last tile of few keys."""
    kw = forms_of(form, Hq)
    D = 64 if fmt == "fp32" else 128
    x = Batch(fmt, D, Hq, H, [0, 333, 3], [299, 250, 131], "chain:299", staged=staged, seed=7)
    rng = np.random.default_rng(0)
    rows = {(b, int(i)) for b in range(3) for i in (0, 1, 127, 128, x.n[b], *rng.integers(0, 131, 5))}
    for depth in (None, ints(np.tile(np.arange(300), (3, 1)))):
        out = x.run(ver, depth=depth, **as_call(kw))
        assert ver.error() == 0
        x.check(out, depth=False, rows=rows, **kw)
        assert torch.equal(out, x.run(ver, depth=depth, **as_call(kw)))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("form", ["cap", "all"])
@pytest.mark.parametrize("staged", [False, True])
def test_forms_of_large_trees(ver, fmt, form, staged):
    """Trees of more entries than a tile: places do not follow one another, rows of all blocks."""
    kw = forms_of(form, 8)
    x = Batch(fmt, 128, 8, 2, [0, 100, 513], [179, 60, 140], "random:179", staged=staged, seed=9, trees=range(3))
    out = x.run(ver, depth=ints(x.depth), **as_call(kw))
    assert ver.error() == 0
    rng = np.random.default_rng(0)
    x.check(out, rows={(b, int(i)) for b in range(3) for i in (0, 1, 127, 128, x.n[b], *rng.integers(0, 180, 9))}, **kw)


@pytest.mark.parametrize("fmt,D", [("bf16", 128), ("e4m3", 64), ("fp32", 64)])
def test_what_a_window_leaves_out_may_be_anything(ver, fmt, D):
    """NaN and infinities outside the window do not reach a row, inside they do."""
    S, W0 = [300, 140], 60
    x = Batch(fmt, D, 4, 2, S, [6, 6], "binary:2", seed=3, trees=[0, 0])
    clean = x.run(ver, depth=ints(x.depth), window=W0)
    spoiled = {0: 300 - W0 + 2, 1: 140 - W0}  # seen by the rows at depths 0 and 1 of request 0; of request 1 by none
    for b, p in spoiled.items():
        for j in (p, 3):
            x.kv[x.table[b, j // 16], 1, :, :, j % 16] = poison(fmt, (2, 2), D)
    out = x.run(ver, depth=ints(x.depth), window=W0)
    assert ver.error() == 0
    for i in range(7):
        assert torch.isnan(out[0, i]).all() if x.depth[0, i] <= 1 else torch.equal(out[0, i], clean[0, i])
    assert torch.equal(out[1], clean[1])


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "fp32"])
def test_rows_that_see_nothing_are_zero(ver, fmt):
    x = Batch(fmt, 64, 4, 2, [0, 50], [4, 4], "chain:4", seed=5)
    x.bits[0, 2] = False      # an empty mask over no cached positions
    x.bits[1, 3] = False      # and under a window that ends before the row
    out = x.run(ver, depth=ints(x.depth), window=3, softcap=5.0)
    assert ver.error() == 0
    assert not out[0, 2].any() and not out[1, 3].any()
    x.check(out, window=3, softcap=5.0)


def test_extreme_scores_and_caps(ver):
    """Scores far past the cap, tiny and huge caps, negative and zero scales."""
    for fmt, D in (("bf16", 128), ("e4m3", 128), ("fp32", 64)):
        for cap, scale in ((1e-3, None), (50.0, 40.0), (1e6, None), (30.0, -0.2), (5.0, 0.0)):
            x = Batch(fmt, D, 4, 2, [200, 17], [3, 3], "chain:3", seed=11, size=3.0)
            out = x.run(ver, softcap=cap, scale=scale)
            assert ver.error() == 0
            got, want = f64(out), f64(x.run(ver, scale=scale))
            if cap == 1e6:  # as good as none: s^3 / (3 cap^2) is below 1e-7
                assert np.abs(got - want).max() <= 2.0 ** -7 * np.abs(want).max()
            x.check(out, softcap=cap, scale=scale, depth=False)


def test_depths_out_of_range_count_as_the_nearest(ver):
    x = Batch("bf16", 128, 4, 1, [90], [7], "random:7", seed=2)
    d = x.depth.copy()
    d[0, 3], d[0, 5] = -4, 1000
    a = x.run(ver, depth=ints(d), window=30, slopes=torch.tensor(some_slopes(4), device=DEV))
    d[0, 3], d[0, 5] = 0, 7
    b = x.run(ver, depth=ints(d), window=30, slopes=torch.tensor(some_slopes(4), device=DEV))
    assert torch.equal(a, b) and ver.error() == 0


# --------------------------------------------------------------------------- #
# shared prefixes
# --------------------------------------------------------------------------- #
def grouped(ver, x, least=1):
    g = ver.prefix_groups(ints(x.table), ints(x.S), x.BS, least=least)
    length, members = E.prefix_groups(x.table, x.S, x.BS, least)
    np.testing.assert_array_equal(g["length"].cpu().numpy(), length)
    np.testing.assert_array_equal(g["members"].cpu().numpy(), members)
    return g


SHARED = [  # fmt, D, Hq, H, BS, tree, staged, prefixes' blocks, S past them, groups
    ("bf16", 128, 8, 2, 16, "chain:0", False, 20, [1, 0, 37, 300], [4]),
    ("bf16", 128, 28, 4, 16, "chain:4", True, 17, [0, 31, 16, 3, 7, 1, 200, 14], [4, 4]),
    ("e4m3", 128, 8, 2, 16, "binary:3", True, 33, [5, 0, 140, 9, 260, 77], [3, 1, 2]),
    ("e4m3", 64, 8, 8, 8, "random:9", False, 40, [5, 0, 140, 9], [2, 2]),
    ("bf16", 64, 16, 2, 64, "binary:2", True, 5, list(range(0, 66, 3)), [22]),
    ("bf16", 128, 32, 8, 32, "random:20", True, 9, [1, 2, 3], [1, 2]),
    ("bf16", 128, 16, 4, 16, "binary:2", True, 30, [4 + 37 * x % 300 for x in range(24)], [8, 8, 8]),  # own keys of many tiles
    ("e4m3", 128, 16, 4, 16, "binary:2", False, 30, [4 + 37 * x % 300 for x in range(16)], [8, 8]),
    ("bf16", 128, 4, 4, 16, "chain:0", True, 8, [40, 50, 0, 1, 2, 3, 4], [2, 1, 4]),
    ("bf16", 128, 16, 2, 16, "random:40", True, 20, [5, 150, 0, 9], [3, 1]),       # more than 128 rows a request
    ("e4m3", 128, 32, 4, 8, "random:40", False, 50, [5, 260, 0, 9], [4]),          # more than 256
    ("bf16", 128, 2, 2, 16, "random:150", True, 9, [5, 60, 0, 9], [3, 1]),         # entries of more than a tile
    ("e4m3", 64, 2, 1, 16, "random:150", True, 9, [5, 60], [2]),
    ("bf16", 64, 4, 4, 16, "chain:0", False, 9, [3 * (x % 17) for x in range(80)], [70, 1, 9]),  # one row a head, many members
    ("fp32", 64, 4, 4, 16, "chain:5", True, 9, [5, 6, 7], [3]),
    ("bf16", 80, 6, 3, 24, "chain:2", True, 6, [5, 6, 7], [3])]


def shared_batch(fmt, D, Hq, H, BS, tree, staged, blocks, own, sizes, **kw):
    common = sum(([0] + [blocks] * (m - 1) for m in sizes), [])
    N = len(W.tree_shape(tree, np.random.default_rng(0)))
    n = [N if b % 3 != 1 else N // 2 for b in range(len(own))]
    return Batch(fmt, D, Hq, H, [blocks * BS + x for x in own], n, tree, staged=staged, BS=BS, common=common,
                 seed=len(own) + D, **kw)


@pytest.mark.parametrize("case", SHARED, ids=lambda c: f"{c[0]}-{c[1]}-{c[5]}")
@pytest.mark.parametrize("form", [None, "cap", "all"])
def test_shared_prefixes(ver, case, form):
    x = shared_batch(*case)
    kw = {} if form is None else forms_of(form, x.Hq)
    if form == "all":
        del kw["window"]
    g = grouped(ver, x)
    out = x.run(ver, depth=ints(x.depth), groups=g, **as_call(kw))
    assert ver.error() == 0
    x.check(out, **kw)
    assert torch.equal(out, x.run(ver, depth=ints(x.depth), groups=g, **as_call(kw)))


def test_a_window_reads_every_requests_own_blocks(ver):
    x = shared_batch(*SHARED[1])
    a = x.run(ver, depth=ints(x.depth), window=100, groups=grouped(ver, x))
    assert torch.equal(a, x.run(ver, depth=ints(x.depth), window=100)) and ver.error() == 0


def test_lengths_inside_a_block_and_no_groups(ver):
    """A shared length that ends inside a block, one past a member's cache, none at all."""
    x = shared_batch("bf16", 128, 8, 2, 16, "chain:3", True, 20, [1, 2, 3, 4], [4])
    for length in ([317] * 4, [16] * 4, [15] * 4, [0] * 4):
        out = x.run(ver, groups=dict(length=ints(length), members=ints([4, 0, 0, 0] if length[0] else [0] * 4)))
        assert ver.error() == 0
        x.check(out, depth=False)


def test_groups_that_cannot_be_are_reported(ver):
    x = shared_batch("bf16", 128, 8, 2, 16, "chain:3", True, 20, [1, 2, 3, 4], [4])
    for length, members in (([320] * 4, [5, 0, 0, 0]), ([320] * 4, [0, 4, 0, 0]), ([320, 320, 160, 320], [4, 0, 0, 0]),
                            ([320] * 4, [0, 0, 0, 0]), ([320] * 4, [3, 0, 0, 0]), ([320] * 4, [4, 0, 2, 0]),
                            ([320] * 4, [-1, 0, 0, 0]), ([320] * 4, [2 ** 31 - 1, 0, 0, 0])):
        x.run(ver, groups=dict(length=ints(length), members=ints(members)))
        assert ver.error() == binding.SV_ERR_STATE, (length, members)
    out = x.run(ver, groups=dict(length=ints([10 ** 6, -5, 400, 0]), members=ints([0, 0, 0, 0])))  # none
    assert ver.error() == 0
    x.check(out, depth=False)


def test_more_requests_than_a_kernels_threads(ver):
    """Groups that cross the 1024 requests at which the list's kernel goes on, the largest lots."""
    x = shared_batch("bf16", 64, 2, 1, 16, "chain:1", True, 8, [(7 * b) % 40 for b in range(1100)], [3, 1000, 40, 1, 56])
    g = grouped(ver, x)
    out = x.run(ver, groups=g)
    assert ver.error() == 0
    rng = np.random.default_rng(0)
    some = {0, 2, 3, 1002, 1003, 1023, 1024, 1042, 1043, 1044, 1099, *rng.integers(0, 1100, 60).tolist()}
    x.check(out, depth=False, rows={(b, i) for b in some for i in (0, 1)})


@pytest.mark.parametrize("fmt,staged", [("bf16", True), ("bf16", False), ("e4m3", True), ("e4m3", False)])
def test_special_values_of_one_request_do_not_reach_the_others(ver, fmt, staged):
    """Own positions and entries of requests lie side by side in a tile."""
    x = shared_batch(fmt, 128, 8, 2, 16, "chain:3", staged, 20, [40, 2, 33, 4], [4])
    g = grouped(ver, x)
    clean = x.run(ver, groups=g)
    p = 20 * 16 + 7
    x.kv[x.table[2, p // 16], 1, :, :, p % 16] = poison(fmt, (2, 2), 128)
    out = x.run(ver, groups=g)
    assert ver.error() == 0
    for b in (0, 1, 3):
        assert torch.equal(out[b], clean[b])
    assert torch.isnan(out[2, :x.n[2] + 1]).all()
    if staged:  # an entry of request 0, seen by the rows from it on
        x = shared_batch(fmt, 128, 8, 2, 16, "chain:3", staged, 20, [40, 2, 33, 4], [4])
        x.stage[0, 2, 1] = poison(fmt, (2, 2), 128)
        out = x.run(ver, groups=g)
        assert ver.error() == 0
        assert torch.equal(out[1:], clean[1:]) and torch.equal(out[0, :2], clean[0, :2]) and torch.isnan(out[0, 2:]).all()


@pytest.mark.parametrize("case", [("bf16", 128, 8, 2, 16, "chain:30", True, 20, [40, 2, 33, 4], [1, 2, 1]),
                                  ("e4m3", 128, 8, 2, 16, "chain:3", True, 20, [40, 2, 33, 4], [4])], ids=["bf16", "e4m3"])
def test_queries_past_a_requests_entries_may_be_anything(ver, case):
    """They are read as zeros: neither the outputs nor their last bits depend on them."""
    x = shared_batch(*case)
    g = grouped(ver, x)
    one = dict(length=g["length"].clone(), members=g["members"].clone())
    for groups in (g, one, None):
        want = x.run(ver, groups=groups, softcap=3.0)
        keep = x.q.clone()
        for bad in (float("nan"), 1e30, -float("inf")):
            for b in range(x.B):
                x.q[b, x.n[b] + 1:] = bad
            assert torch.equal(x.run(ver, groups=groups, softcap=3.0), want)
        x.q.copy_(keep)
    assert ver.error() == 0


def test_special_values_in_a_prefix_reach_its_rows_alone(ver):
    x = shared_batch("bf16", 128, 8, 2, 16, "chain:3", True, 20, [1, 2, 3, 4], [2, 2])
    g = grouped(ver, x)
    clean = x.run(ver, groups=g)
    x.kv[x.table[0, 3], 1, 1, :, 5] = float("nan")  # a value of the first group's prefix
    out = x.run(ver, groups=g)
    assert torch.isnan(out[:2]).all(-1)[(torch.arange(4, device=DEV) <= ints(x.n)[:2, None])].all()
    assert torch.equal(out[2:], clean[2:]) and ver.error() == 0


def test_captured_and_on_another_stream(ver):
    x = shared_batch(*SHARED[1])
    y = shared_batch(*SHARED[2])
    gx, gy = grouped(ver, x), grouped(ver, y)
    kw = dict(softcap=20.0)
    wx, wy = x.run(ver, groups=gx, **kw), y.run(ver, groups=gy)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    words = [torch.tensor(E.pack(z.bits).view(np.int32), device=DEV) for z in (x, y)]
    args = [(z.q, z.kv, ints(z.table), ints(z.S)) for z in (x, y)]
    more = [dict(layer=1, stage=z.stage, mask=w, n_nodes=ints(z.n)) for z, w in zip((x, y), words)]
    torch.cuda.synchronize()
    for _ in range(5):  # two at once
        a = ver.tree_attention(*args[0], **more[0], groups=gx, stream=s1, **kw)
        b = ver.tree_attention(*args[1], **more[1], groups=gy, stream=s2)
        torch.cuda.synchronize()
        assert torch.equal(a, wx) and torch.equal(b, wy)
    out = torch.zeros_like(x.q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g2 = ver.prefix_groups(args[0][2], args[0][3], x.BS, least=1)
        ver.tree_attention(*args[0], **more[0], groups=g2, out=out, **kw)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, wx)
    assert ver.error() == 0


# --------------------------------------------------------------------------- #
# groups
# --------------------------------------------------------------------------- #
@pytest.mark.parametrize("B,width,BS,least", [(1, 3, 16, 1), (2, 1, 16, 128), (7, 40, 16, 128), (300, 70, 8, 100),
                                              (1100, 3, 1, 1), (5, 3000, 16, 128), (64, 12, 16, 0), (33, 9, 4, 10 ** 9)])
def test_prefix_groups(ver, B, width, BS, least):
    rng = np.random.default_rng(B + width)
    table = rng.integers(0, 10 ** 6, (B, width)).astype(np.int32)
    lens = rng.integers(0, width * BS + 1, B)
    for b in range(1, B):
        c = int(rng.integers(0, width + 1)) if rng.random() < 0.8 else 0
        c = width if rng.random() < 0.3 else c
        table[b, :c] = table[b - 1, :c]
        if rng.random() < 0.7:
            lens[b] = max(lens[b], lens[b - 1])
        if rng.random() < 0.1:
            table[b - 1:b + 1, int(rng.integers(0, width))] = -1
    out = dict(length=torch.full((B,), -9, dtype=torch.int32, device=DEV), members=torch.full((B,), -9, dtype=torch.int32, device=DEV))
    got = ver.prefix_groups(ints(table), ints(lens), BS, least=least, out=out)
    length, members = E.prefix_groups(table, lens, BS, least)
    np.testing.assert_array_equal(got["length"].cpu().numpy(), length)
    np.testing.assert_array_equal(got["members"].cpu().numpy(), members)
    assert ver.error() == 0
    again = ver.prefix_groups(ints(table), ints(lens), BS, least=least, stream=torch.cuda.Stream())
    torch.cuda.synchronize()
    assert torch.equal(again["length"], got["length"]) and torch.equal(again["members"], got["members"])


def test_prefix_groups_of_bad_lengths(ver):
    table = ints([[1, 2], [1, 2], [1, 2], [1, 2]])
    for bad in (33, -1):
        got = ver.prefix_groups(table, ints([32, 32, bad, 32]), 16, least=1)
        assert ver.error() == binding.SV_ERR_STATE
        assert got["length"].tolist() == [32, 32, 0, 0] and got["members"].tolist() == [2, 0, 0, 0]
    empty = ver.prefix_groups(ints(np.zeros((0, 4))), ints([]), 16)
    assert empty["length"].numel() == 0 and ver.error() == 0
    none = ver.prefix_groups(ints(np.zeros((3, 0))), ints([0, 0, 0]), 16)
    assert none["members"].tolist() == [0, 0, 0] and ver.error() == 0


def test_refusals(ver):
    x = shared_batch("bf16", 128, 8, 2, 16, "chain:3", True, 2, [1, 2], [2])
    z = ints([0, 0])
    for kw in (dict(softcap=0.0), dict(softcap=-1.0), dict(softcap=float("nan")), dict(softcap=1e30), dict(window=0),
               dict(window=-3), dict(window=2 ** 31), dict(slopes=torch.zeros(7, device=DEV)),
               dict(slopes=torch.zeros(8, device=DEV, dtype=torch.bfloat16)), dict(slopes=torch.zeros(16, device=DEV)[::2]),
               dict(depth=ints([[0, 1], [0, 1]])), dict(depth=torch.zeros(2, 4, device=DEV)),
               dict(groups=dict(length=z, members=None)), dict(groups=dict(length=z[:1], members=z)),
               dict(groups=dict(length=z.long(), members=z))):
        with pytest.raises((ValueError, binding.SvError)):
            x.run(ver, **kw)
    for args in ((x.table[0], z, 16), (x.table, z, 0), (x.table, z[:1], 16)):
        with pytest.raises((ValueError, binding.SvError)):
            ver.prefix_groups(ints(args[0]), *args[1:])
    with pytest.raises(ValueError):
        ver.prefix_groups(ints(x.table), z, 16, out=dict(length=z))
    torch.cuda.synchronize()
    assert ver.error() == 0
