"""sv_tree_mask, kv_append / kv_read, sv_tree_attention and sv_adjust_logits
against the fp64 definitions, at the sizes and masks where they can go wrong.

Bounds, derived before any run (u = 2^-24, the fp32 rounding unit):
  bf16 result            half an ulp of an 8-bit significand: 2^-8 |y|
  rotation               two products and a sum on fp32 cos / sin: 4 u (|x1| + |x2|)
  e4m3                   half a step: 2^-4 |x|, or 2^-10 scale below the normal range
  attention, fp32        scores: (D + 3) u times the largest sum |q||k| scale; weights and
                         output: the sums over n keys, (n + 16) u each; in units of sum p |v|
  attention, bf16        weights rounded to 8 bits 2^-8 and the fp32 terms below 2^-10, in units
                         of sum p |v|, and the output's own 2^-8 |o|
  logits                 six roundings: 6 u times the sum of the terms' sizes
"""

import os

import numpy as np
import pytest
import torch

from oracle import entries as E
from oracle import kvcache as KC
from speculative_decoding_verification_07_gb300 import binding, rope
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


def words(a):
    return torch.tensor(np.ascontiguousarray(a).view(np.int32), device=DEV)


def f64(t):
    return t.detach().cpu().numpy() if t.dtype == torch.uint8 else t.detach().double().cpu().numpy()


def parents(shape, seed=0):
    return W.tree_shape(shape, np.random.default_rng(seed))


def row_len(fmt, D):
    return D + E.TAIL if fmt == "e4m3" else D


def random_entries(shape, fmt, D, seed, size=1.0):
    """Random entry rows [..., row] on the GPU."""
    g = torch.Generator(DEV).manual_seed(seed)
    x = torch.randn(*shape, D, generator=g, device=DEV) * size
    if fmt != "e4m3":
        return x.to(TORCH[fmt])
    out = torch.zeros(*shape, D + E.TAIL, dtype=torch.uint8, device=DEV)
    e = torch.randint(-9, -5, tuple(shape), generator=g, device=DEV).float()
    out[..., :D] = (x * 80).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    out[..., D:D + 4] = torch.exp2(e).unsqueeze(-1).view(torch.uint8)
    return out


def poison(fmt, shape, D):
    """Entry rows that ruin whatever they enter: NaN values (and a NaN scale)."""
    if fmt == "e4m3":
        return torch.full((*shape, D + E.TAIL), 0xFF, dtype=torch.uint8, device=DEV)
    return torch.full((*shape, D), float("nan"), dtype=TORCH[fmt], device=DEV)


def tables(lens, BS, rng, extra=3):
    """Random block tables covering the lengths, and the pool's size."""
    n = [-(-int(x) // BS) for x in lens]
    order = rng.permutation(sum(n) + extra)
    t = np.full((len(n), max(1, max(n))), -1, np.int32)
    at = 0
    for b, m in enumerate(n):
        t[b, :m] = order[at:at + m]
        at += m
    return t, sum(n) + extra


# --------------------------------------------------------------------------- #
# tree masks
# --------------------------------------------------------------------------- #
@pytest.mark.parametrize("shape,B", [("chain:0", 3), ("chain:1", 1), ("binary:3", 64), ("random:31", 5),
                                     ("random:32", 5), ("wide:7,5", 4), ("random:300", 3), ("chain:1100", 1)])
def test_tree_mask(ver, shape, B):
    rng = np.random.default_rng(7)
    N = len(parents(shape))
    par = np.array([parents(shape, s) for s in range(B)], np.int32).reshape(B, N)
    n = rng.integers(-1, N + 1, B)
    n[0] = N
    for nn, ld in ((None, None), (n, -(-(N + 1) // 32) + 2)):
        out = None if ld is None else dict(mask=torch.full((B, N + 1, ld), -1, dtype=torch.int32, device=DEV),
                                           depth=torch.full((B, N + 1), -7, dtype=torch.int32, device=DEV))
        got = ver.tree_mask(ints(par), n_nodes=None if nn is None else ints(nn), out=out)
        assert ver.error() == 0
        for b in range(B):
            bits, depth = E.ancestors(par[b], N if nn is None else int(nn[b]))
            np.testing.assert_array_equal(got["mask"][b].cpu().numpy().view(np.uint32), E.pack(bits, got["mask"].shape[2]))
            np.testing.assert_array_equal(got["depth"][b].cpu().numpy(), depth)


def test_tree_mask_bad_parents_are_reported(ver):
    got = ver.tree_mask(ints([[0, 5, 1]]))
    assert ver.error() == binding.SV_ERR_STATE
    np.testing.assert_array_equal(got["depth"].cpu().numpy(), [[0, 1, 1, 2]])  # node 2 under the root
    ver.tree_mask(ints([[0, 5, 1]]), n_nodes=ints([1]))  # not one of the request's nodes
    assert ver.error() == 0


# --------------------------------------------------------------------------- #
# entries
# --------------------------------------------------------------------------- #
@pytest.mark.parametrize("dtype,fmt", [("bf16", "bf16"), ("bf16", "e4m3"), ("fp32", "fp32"), ("fp32", "e4m3"),
                                       ("bf16", "fp32"), ("fp32", "bf16")])
@pytest.mark.parametrize("D,Hq,H,rot,pairs,BS,staged", [
    (128, 32, 8, 128, False, 16, True), (128, 28, 4, 64, True, 16, False), (64, 4, 4, 64, False, 1, False),
    (80, 6, 3, 32, False, 24, False), (16, 4, 2, 0, False, 16, True), (256, 2, 1, 256, True, 16, False),
    (96, 5, 5, 24, False, 16, True), (64, 3, 1, 6, True, 7, False)])
def test_append_and_read(ver, dtype, fmt, D, Hq, H, rot, pairs, BS, staged):
    rng = np.random.default_rng(D + Hq)
    B, R, L = 5, 9, 3
    par = np.array([parents("random:8", s) for s in range(B)], np.int32)
    n = np.array([8, 0, -1, 5, 3])
    S = np.array([0, 700, 31, 15, 129])
    depth = np.stack([E.ancestors(par[b], 8)[1] for b in range(B)])
    g = torch.Generator(DEV).manual_seed(D)
    qkv = torch.randn(B, R, Hq + 2 * H, D, generator=g, device=DEV) * torch.exp2(
        torch.randint(-8, 9, (B, R, 1, 1), generator=g, device=DEV).float())
    qkv = qkv.to(TORCH[dtype])
    qkv[0, 1, Hq] = 0                      # an all-zero key row
    keep = qkv.clone()
    q, k, v = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + H], qkv[:, :, Hq + H:]
    rows = row_len(fmt, D)
    if staged:
        data = torch.full((B, R, L, 2, H, rows), 77, dtype=TORCH[fmt], device=DEV)
        place = dict(stage=data)
    else:
        t, nb = tables(S + R, BS, rng)
        data = torch.full((nb, L, 2, H, BS, rows), 77, dtype=TORCH[fmt], device=DEV)
        place = dict(kv=data, block_table=ints(t))
    freq = rope.rope_frequencies(rot) if rot else None
    table = rope.rope_table(800, freq) if rot else None
    q_out = torch.full((B, R, Hq, D), 5.0, dtype=TORCH[dtype], device=DEV)
    ver.kv_append(k, v, ints(S), layer=1, q=q, q_out=q_out, rope=table, interleaved=pairs, depth=ints(depth),
                  n_nodes=ints(n), **place)
    out_t = torch.bfloat16 if dtype == "bf16" else torch.float32
    back = torch.full((B, R, 2, H, D), 5.0, dtype=out_t, device=DEV)
    ver.kv_read(back, ints(S), layer=1, n_nodes=ints(n), **place)
    assert ver.error() == 0
    assert torch.equal(qkv, keep)
    x, qo, bk, raw = f64(keep), f64(q_out), f64(back), f64(data)
    written = np.zeros(raw.shape, bool)
    half_ulp = 2.0 ** -8 if dtype == "bf16" else U
    for b in range(B):
        for i in range(R):
            if i > n[b]:
                assert not qo[b, i].any() and not bk[b, i].any()
                continue
            pos = S[b] + depth[b, i]
            y, size = x[b, i].copy(), np.zeros_like(x[b, i])
            if rot:
                c, s = np.cos(pos * freq.numpy()), np.sin(pos * freq.numpy())
                y[:Hq + H] = E.rotate(x[b, i, :Hq + H], c, s, pairs)
                size[:Hq + H] = E.rotate(np.abs(x[b, i, :Hq + H]), np.ones_like(c), -np.ones_like(c), pairs)
                size[:Hq + H] += E.rotate(np.abs(x[b, i, :Hq + H]), np.ones_like(c), np.ones_like(c), pairs)
                size = np.abs(size)  # 2 |x1| on the first of a pair, 2 |x2| on the second
                size = np.broadcast_to(size.max(-1, keepdims=True), size.shape)
            err = 4 * U * size
            assert (np.abs(qo[b, i] - y[:Hq]) <= half_ulp * np.abs(y[:Hq]) + err[:Hq]).all()
            at = (b, i, 1) if staged else (t[b, (S[b] + i) // BS], 1, slice(None), slice(None), (S[b] + i) % BS)
            written[at] = True
            rowsv = raw[at]  # [2, H, row]
            want = np.stack([y[Hq:Hq + H], y[Hq + H:]])
            e2 = np.stack([err[Hq:Hq + H], err[Hq + H:]])
            val = E.decode(rowsv, fmt, D)
            if fmt == "e4m3":
                scale = np.ascontiguousarray(rowsv[..., D:D + 4]).view(np.float32)[..., 0].astype(np.float64)
                assert not rowsv[..., D + 4:].any()
                if rot:  # a maximum that rounds across the boundary may take the other scale
                    ref = E.e4m3_scale(want)
                    assert ((scale == ref) | (np.abs(np.abs(want).max(-1) / scale / 448 - 1) < 1e-5)
                            | (np.abs(np.abs(want).max(-1) / scale / 224 - 1) < 1e-5)).all()
                else:
                    np.testing.assert_array_equal(scale, E.e4m3_scale(want))
                    np.testing.assert_array_equal(val, E.e4m3_round(want / scale[..., None]) * scale[..., None])
                tol = np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10 * scale[..., None]) + 2 * e2
            else:
                tol = (2.0 ** -8 if fmt == "bf16" else U) * np.abs(want) + e2
            assert (np.abs(val - want) <= tol).all()
            read_ulp = 2.0 ** -8 if dtype == "bf16" else 0.0
            assert (np.abs(bk[b, i] - val) <= read_ulp * np.abs(val)).all()
    assert (raw[~written] == 77).all()  # nothing else was touched


def test_append_special_values(ver):
    """Infinities, NaN, subnormals and the scale's boundary, in 8 bits."""
    D = 32
    x = torch.zeros(1, 6, 1, D, device=DEV)
    x[0, 0, 0, 3] = 448.0
    x[0, 1, 0, 3] = 448.0001
    x[0, 2, 0, :2] = torch.tensor([1e-40, -3e-39])
    x[0, 3, 0, :3] = torch.tensor([float("nan"), 7.0, -3.0])
    x[0, 4, 0, :3] = torch.tensor([float("inf"), 1.0, -float("inf")])
    x[0, 5, 0, :2] = torch.tensor([3e38, -1e38])
    stage = torch.zeros(1, 6, 1, 2, 1, D + E.TAIL, dtype=torch.uint8, device=DEV)
    ver.kv_append(x, x, ints([0]), stage=stage)
    out = torch.empty(1, 6, 2, 1, D, device=DEV)
    ver.kv_read(out, ints([0]), stage=stage)
    assert ver.error() == 0
    scale = stage[0, :, 0, 0, 0, D:D + 4].contiguous().view(torch.float32).flatten().tolist()
    assert scale == [1.0, 2.0, 2.0 ** -126, 2.0 ** -6, 2.0 ** 120, 2.0 ** 120]
    y = out[0, :, 1, 0].cpu()
    assert y[0, 3] == 448 and y[1, 3] == 448
    assert torch.isnan(y[3, 0]) and y[3, 1] == 7 and y[3, 2] == -3
    assert y[4, 0] == float("inf") and y[4, 2] == -float("inf") and y[4, 1] == 0
    assert abs(y[5, 0] / 3e38 - 1) < 2 ** -4


def test_append_in_place_and_on_another_stream(ver):
    g = torch.Generator(DEV).manual_seed(3)
    q = torch.randn(3, 4, 8, 128, generator=g, device=DEV).bfloat16()
    k = torch.randn(3, 4, 2, 128, generator=g, device=DEV).bfloat16()
    table = rope.rope_table(64, rope.rope_frequencies(128))
    stage = [torch.zeros(3, 4, 1, 2, 2, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    want = ver.kv_append(k, k, ints([1, 20, 59]), q=q, rope=table, stage=stage[0])
    inplace = q.clone()
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    ver.kv_append(k, k, ints([1, 20, 59]), q=inplace, q_out=inplace, rope=table, stage=stage[1], stream=st)
    torch.cuda.synchronize()
    assert torch.equal(inplace, want) and torch.equal(stage[0], stage[1])
    assert ver.error() == 0


def test_append_out_of_range_is_skipped_and_reported(ver):
    k = torch.ones(2, 3, 1, 64, device=DEV)
    kv = torch.zeros(4, 1, 2, 1, 4, 64, device=DEV)
    t = ints([[0, 1], [2, -1]])
    ver.kv_append(k, k, ints([6, 0]), kv=kv, block_table=t)       # request 0's third entry has no block
    assert ver.error() == binding.SV_ERR_STATE
    assert kv[1, 0, :, :, 2:].eq(1).all() and kv[2, 0, :, :, :3].eq(1).all() and kv.sum() == 2 * 64 * 5
    table = rope.rope_table(2, rope.rope_frequencies(64))
    q = torch.ones(2, 3, 1, 64, device=DEV)
    qo = ver.kv_append(k, k, ints([0, 0]), kv=kv, block_table=t, q=q, rope=table)
    assert ver.error() == binding.SV_ERR_STATE
    assert not qo[:, 2].any() and qo[:, 0].eq(1).all()
    out = torch.full((2, 3, 2, 1, 64), 9.0, device=DEV)
    ver.kv_read(out, ints([6, 0]), kv=kv, block_table=t)
    assert ver.error() == binding.SV_ERR_STATE
    assert not out[0, 2].any()


# --------------------------------------------------------------------------- #
# attention
# --------------------------------------------------------------------------- #
def check_attention(ver, fmt, D, Hq, H, S, n, bits, staged, BS=16, seed=0, L=2, layer=1, scale=None, mask=True,
                    strided=False, size=1.0, bad_rows=()):
    """Random inputs in poisoned surroundings; every row against the definition.
    bad_rows: (request, entry) whose K and V are NaN: rows that see them are NaN."""
    rng = np.random.default_rng(seed)
    B, R = len(S), bits.shape[1]
    S, n = np.asarray(S), np.asarray(n)
    n_ent = np.maximum(n + 1, 0)
    t, nb = tables(S + (0 if staged else n_ent), BS, rng)
    kv = poison(fmt, (nb, L, 2, H, BS), D)
    stage = poison(fmt, (B, R, L, 2, H), D) if staged else None
    K, V = [], []
    for b in range(B):
        e = random_entries((S[b] + n_ent[b], 2, H), fmt, D, seed * 1000 + b, size)
        for (bb, i) in bad_rows:
            if bb == b:
                e[S[b] + i] = poison(fmt, (2, H), D)
        val = E.decode(f64(e), fmt, D)
        K.append(val[:, 0]), V.append(val[:, 1])
        in_cache = S[b] + (0 if staged else n_ent[b])
        if in_cache:
            p = torch.arange(in_cache, device=DEV)
            kv[ints(t[b]).long()[p // BS], layer, :, :, p % BS] = e[:in_cache]
        if staged:
            stage[b, :n_ent[b], layer] = e[S[b]:]
    dt = torch.float32 if fmt == "fp32" else torch.bfloat16
    g = torch.Generator(DEV).manual_seed(seed + 5)
    if strided:  # a slice of a wider projection, and an output of its own
        q = torch.randn(B, R, Hq + 2 * H, D, generator=g, device=DEV).to(dt)[:, :, :Hq]
        out = torch.full((B, R, 2 * Hq, D), 3.0, dtype=dt, device=DEV)[:, :, Hq:]
    else:
        q = torch.randn(B, R, Hq, D, generator=g, device=DEV).to(dt)
        out = torch.full((B, R, Hq, D), 3.0, dtype=dt, device=DEV)
    ver.tree_attention(q, kv, ints(t), ints(S), layer=layer, stage=stage, n_nodes=ints(n), scale=scale, out=out,
                       mask=words(E.pack(bits)) if mask else None)
    assert ver.error() == 0
    again = torch.full_like(out, 4.0)
    ver.tree_attention(q, kv, ints(t), ints(S), layer=layer, stage=stage, n_nodes=ints(n), scale=scale, out=again,
                       mask=words(E.pack(bits)) if mask else None)
    torch.cuda.synchronize()
    assert torch.equal(out.contiguous().view(torch.uint8), again.contiguous().view(torch.uint8))
    got, qd = f64(out), f64(q)
    sc = D ** -0.5 if scale is None else scale
    worst = 0.0
    for b in range(B):
        for i in range(R):
            if i > n[b]:
                assert not got[b, i].any()
                continue
            seen = np.concatenate([np.ones(S[b], bool), bits[b, i, :n[b] + 1]])
            for h in range(Hq):
                kh = h // (Hq // H)
                if any(bb == b and bits[b, i, j] for bb, j in bad_rows):
                    assert np.isnan(got[b, i, h]).all()
                    continue
                o, size_v, size_s = E.attend(qd[b, i, h], K[b][:, kh], V[b][:, kh], seen, sc)
                if fmt == "fp32":
                    tol = (2 * (D + 3) * U * size_s + 2 * (seen.sum() + 16) * U) * size_v
                else:
                    tol = (2.0 ** -8 + 2.0 ** -10) * size_v + 2.0 ** -8 * np.abs(o)
                d = np.abs(got[b, i, h] - o)
                assert (d <= tol).all(), (b, i, h, d.max(), tol[d.argmax()])
                worst = max(worst, float((d / np.maximum(tol, 1e-300)).max()) if size_v.any() else 0.0)
    return worst


def tree_bits(shape, B, n):
    par = [parents(shape, s) for s in range(B)]
    return np.stack([E.ancestors(par[b], len(par[b]))[0] for b in range(B)])


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "fp32"])
@pytest.mark.parametrize("D,Hq,H,shape,S,staged,BS", [
    (128, 8, 2, "binary:3", [0, 1, 15, 16, 17, 127, 128, 129, 300], True, 16),
    (128, 8, 2, "binary:3", [0, 1, 15, 16, 17, 127, 128, 129, 300], False, 16),
    (64, 4, 4, "chain:5", [32, 0, 5], True, 16),
    (64, 14, 2, "random:40", [513, 64, 0], True, 32),
    (128, 28, 4, "random:40", [100, 700], False, 16),
    (128, 32, 8, "chain:0", [777, 0, 1, 2049], False, 16),
    (64, 8, 8, "chain:0", [90, 64, 63], True, 64),
    (128, 4, 1, "wide:4,3", [200, 50], True, 8),
    (64, 4, 2, "binary:2", [77, 300], False, 256),
    (128, 4, 2, "binary:2", [61, 130], True, 1),
    (80, 4, 2, "binary:2", [61, 130], False, 24),
    (256, 2, 1, "chain:3", [70], True, 16),
    (16, 2, 2, "random:70", [40, 9], False, 5),
])
def test_attention(ver, fmt, D, Hq, H, shape, S, staged, BS):
    B, N = len(S), len(parents(shape))
    bits = tree_bits(shape, B, N)
    check_attention(ver, fmt, D, Hq, H, S, np.full(B, N), bits, staged, BS, seed=D + Hq)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "fp32"])
@pytest.mark.parametrize("staged", [True, False])
def test_attention_ragged_and_empty_rows(ver, fmt, staged):
    """Requests of any size, none included; masks that leave rows empty; a
    pattern that is no tree."""
    rng = np.random.default_rng(11)
    n = np.array([14, -1, 0, 7, 3, 13])
    S = np.array([0, 40, 0, 0, 260, 128])
    bits = rng.random((6, 15, 15)) < 0.4
    bits[0, 3] = bits[2, 0] = bits[3, 7] = False  # no prefix and an empty mask: zero rows
    bits[4, 2] = False                             # the prefix alone
    check_attention(ver, fmt, 128, 8, 2, S, n, bits, staged, seed=2, strided=True)
    check_attention(ver, fmt, 64, 8, 2, S, n, bits, staged, seed=3, scale=0.37)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "fp32"])
@pytest.mark.parametrize("staged", [True, False])
def test_attention_chain_without_mask(ver, fmt, staged):
    bits = np.repeat(np.tril(np.ones((6, 6), bool))[None], 3, 0)
    check_attention(ver, fmt, 128, 8, 4, [3, 130, 513], [5, 2, 5], bits, staged, seed=4, mask=False)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "fp32"])
@pytest.mark.parametrize("staged", [True, False])
def test_attention_unseen_nan_stays_out(ver, fmt, staged):
    """A branch whose K/V are NaN ruins the rows that see it and no other."""
    bits = tree_bits("binary:3", 2, 14)
    check_attention(ver, fmt, 128, 8, 2, [70, 0], [14, 14], bits, staged, seed=5, bad_rows=[(0, 2), (1, 9)])


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_attention_large_scores(ver, fmt):
    """Scores of hundreds: the running maximum moves and old sums are rescaled."""
    bits = tree_bits("binary:3", 3, 14)
    check_attention(ver, fmt, 128, 8, 2, [700, 129, 2], [14] * 3, bits, True, seed=6, size=6.0, scale=1.0)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_attention_long_and_wide(ver, fmt):
    """Many tiles split over the GPU, more rows than one tile, groups of 7."""
    bits = tree_bits("random:63", 2, 63)
    check_attention(ver, fmt, 128, 28, 4, [9001, 3], [63, 50], bits, True, seed=7)


def test_attention_many_requests(ver):
    rng = np.random.default_rng(9)
    S = rng.integers(0, 60, 300)
    check_attention(ver, "bf16", 64, 4, 2, S, rng.integers(-1, 3, 300), tree_bits("chain:2", 300, 2), True, seed=8)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_attention_past_32_bit_offsets(ver, fmt):
    """Blocks beyond 4 GiB (and 2^32 elements' worth of rows) of the cache."""
    D, H, BS = 128, 8, 16
    nb = (9 << 30) // (2 * H * BS * row_len(fmt, D) * (2 if fmt == "bf16" else 1))
    kv = torch.zeros(nb, 1, 2, H, BS, row_len(fmt, D), dtype=TORCH[fmt], device=DEV)
    e = random_entries((32, 2, H), fmt, D, 1)
    for j, blk in enumerate((nb - 1, nb // 2 + 1)):
        kv[blk, 0] = e[16 * j:16 * j + 16].permute(1, 2, 0, 3)
    q = torch.randn(1, 1, H, D, device=DEV).bfloat16()
    out = ver.tree_attention(q, kv, ints([[nb - 1, nb // 2 + 1]]), ints([31]))
    back = torch.empty(1, 32, 2, H, D, device=DEV)
    ver.kv_read(back, ints([0]), kv=kv, block_table=ints([[nb - 1, nb // 2 + 1]]))
    assert ver.error() == 0
    val = E.decode(f64(e), fmt, D)
    np.testing.assert_array_equal(f64(back)[0], val)
    for h in range(H):
        o, size, _ = E.attend(f64(q)[0, 0, h], val[:, 0, h], val[:, 1, h], np.ones(32, bool), D ** -0.5)
        assert (np.abs(f64(out)[0, 0, h] - o) <= (2.0 ** -8 + 2.0 ** -10) * size + 2.0 ** -8 * np.abs(o)).all()


def test_attention_errors_are_reported(ver):
    q = torch.ones(2, 1, 2, 64, device=DEV).bfloat16()
    kv = torch.ones(3, 1, 2, 2, 16, 64, device=DEV).bfloat16()
    out = ver.tree_attention(q, kv, ints([[0], [1]]), ints([16, 3]))  # request 0's entry is past its table
    assert ver.error() == binding.SV_ERR_STATE
    assert not out[0].any() and out[1].eq(1).all()
    out = ver.tree_attention(q, kv, ints([[0], [1]]), ints([-1, 3]))
    assert ver.error() == binding.SV_ERR_STATE
    assert not out[0].any() and out[1].eq(1).all()
    ver.tree_attention(q, kv, ints([[7], [1]]), ints([2, 3]))  # a block outside the pool
    assert ver.error() == binding.SV_ERR_STATE
    out = ver.tree_attention(q, kv, ints([[0], [1]]), ints([2, 3]), n_nodes=ints([1, 0]))
    assert ver.error() == binding.SV_ERR_STATE
    assert not out[0].any() and out[1].eq(1).all()
    out = ver.tree_attention(q, kv, ints([[2], [1]]), ints([2, 3]))
    assert ver.error() == 0 and out.eq(1).all()


def test_attention_on_another_stream_and_reused_workspace(ver):
    """Different shapes back to back on one workspace, on a side stream."""
    st = torch.cuda.Stream()
    g = torch.Generator(DEV).manual_seed(1)
    jobs = []
    for B, S, D in ((1, 4000, 128), (9, 100, 64), (3, 2000, 128)):
        kv = torch.randn(B * 300, 1, 2, 2, 16, D, generator=g, device=DEV).bfloat16()
        t = torch.randperm(B * 300, generator=g, device=DEV).int().reshape(B, 300)
        q = torch.randn(B, 2, 8, D, generator=g, device=DEV).bfloat16()
        jobs.append((q, kv, t, ints([S] * B)))
    first = [ver.tree_attention(*j) for j in jobs]
    torch.cuda.synchronize()
    outs = [torch.empty_like(f) for f in first]
    for _ in range(2):
        for j, o in zip(jobs, outs):
            ver.tree_attention(*j, out=o, stream=st)
    torch.cuda.synchronize()
    for f, o in zip(first, outs):
        assert torch.equal(f, o)
    assert ver.error() == 0


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_staged_tree_attention_equals_committed_cache(ver, fmt):
    """A tree's path attended from the stage, then committed with
    kv_commit_tree: attending it from the cache gives the same rows."""
    D, H, Hq, BS, B = 128, 2, 8, 16, 4
    par = parents("binary:3")
    N, R = len(par), len(par) + 1
    bits, depth = E.ancestors(par, N)
    S = np.array([5, 30, 14, 47])
    rp = KC.BlockPool(40, BS)
    t = np.full((B, 5), -1, np.int32)
    rp.reserve(S * 0, S + 3, t)
    kv = random_entries((40, 1, 2, H, BS), fmt, D, 1)
    g = torch.Generator(DEV).manual_seed(2)
    qkv = torch.randn(B, R, Hq + 2 * H, D, generator=g, device=DEV).bfloat16()
    stage = torch.zeros(B, R, 1, 2, H, row_len(fmt, D), dtype=TORCH[fmt], device=DEV)
    table = rope.rope_table(64, rope.rope_frequencies(D))
    m = ver.tree_mask(ints([par] * B))
    q = ver.kv_append(qkv[:, :, Hq:Hq + H], qkv[:, :, Hq + H:], ints(S), stage=stage, q=qkv[:, :, :Hq], rope=table,
                      depth=m["depth"])
    o1 = ver.tree_attention(q, kv, ints(t), ints(S), stage=stage, mask=m["mask"])
    leaf = [7, 10, 14, 12]
    paths = [[j for j in range(1, N + 1) if bits[leaf[b], j]] for b in range(B)]
    path = np.full((B, N), -1, np.int32)
    for b in range(B):
        path[b, :3] = paths[b]
    binding.kv_commit_tree(ver.handle, ints([3] * B), ints(path), ints(S), ints(t), BS, 40, stage, kv, 3)
    sel = torch.tensor([[0] + paths[b] for b in range(B)], device=DEV)
    qs = q.gather(1, sel[:, :, None, None].expand(B, 4, Hq, D)).contiguous()
    o2 = ver.tree_attention(qs, kv, ints(t), ints(S))
    assert ver.error() == 0
    want = o1.gather(1, sel[:, :, None, None].expand(B, 4, Hq, D))
    # the same sums in another order of keys: two bf16 outputs, weights of 8 bits each
    assert (o2.float() - want.float()).abs().max() <= 2.0 ** -7 * 4
    back = torch.empty(B, 4, 2, H, D, device=DEV)
    ver.kv_read(back, ints(S), kv=kv, block_table=ints(t))
    staged = torch.empty(B, R, 2, H, D, device=DEV)
    ver.kv_read(staged, ints(S), stage=stage)
    assert torch.equal(back, staged.gather(1, sel[:, :, None, None, None].expand(B, 4, 2, H, D)))


# --------------------------------------------------------------------------- #
# logits
# --------------------------------------------------------------------------- #
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V,shape,B,H,nb", [(1024, "chain:5", 3, 37, 5), (1, "chain:0", 2, 3, 1), (31, "random:9", 4, 50, 9),
                                            (4093, "binary:3", 3, 200, 40), (32000, "random:14", 5, 1500, 64),
                                            (8195, "chain:40", 2, 0, 0), (128256, "binary:2", 2, 1500, 300)])
def test_adjust_logits(ver, dtype, V, shape, B, H, nb):
    rng = np.random.default_rng(V + B)
    par = [parents(shape, s) for s in range(B)]
    N, R = len(par[0]), len(par[0]) + 1
    bits = np.stack([E.ancestors(p, N)[0] for p in par])
    n = rng.integers(-1, N + 1, B)
    n[0] = N
    ld = -(-V // 8) * 8 + 16
    g = torch.Generator(DEV).manual_seed(V)
    logits = (torch.randn(B, R, ld, generator=g, device=DEV) * 3).to(TORCH[dtype])
    if V > 100:
        logits[0, 0, :4] = torch.tensor([float("nan"), float("-inf"), float("inf"), 0.0])
    hist = rng.integers(-2, V + 3, (B, H)) if H else np.zeros((B, 0), np.int64)
    hist[:, :H // 3] = rng.integers(0, min(V, 12), (B, H // 3))  # repeats
    toks = rng.integers(0, min(V, 40), (B, N))
    ids = rng.integers(-1, V + 1, (B, nb))
    vals = rng.standard_normal((B, nb)).astype(np.float32) * 4
    if nb >= 5:
        ids[:, 1:5] = 3 % V   # one token named four times
        vals[0, 0] = -np.inf
    rep, pres, freq = rng.uniform(0.7, 2, B), rng.uniform(-0.5, 1, B), rng.uniform(0, 0.6, B)
    allowed = rng.random((B, R, V)) < 0.7
    allowed[0, R - 1] = False
    f32 = lambda a: torch.tensor(a, dtype=torch.float32, device=DEV)  # noqa: E731
    rep, pres, freq = (f32(a) for a in (rep, pres, freq))
    for use_mask, use_allowed, place in ((True, True, "new"), (False, False, "in"), (True, True, "in")):
        src = logits.clone()
        out = src if place == "in" else torch.full((B, R, ld + 8), 9.0, dtype=TORCH[dtype], device=DEV)
        kw = dict(bias_ids=ints(ids), bias_values=f32(vals)) if nb else {}
        ver.adjust_logits(src, V=V, out=None if place == "in" else out, history=ints(hist) if H else None,
                          tokens=ints(toks), mask=words(E.pack(bits)) if use_mask else None, n_nodes=ints(n),
                          rep_penalty=rep, presence=pres, frequency=freq,
                          allowed=words(E.pack(allowed)) if use_allowed else None, **kw)
        assert ver.error() == 0
        got, x = f64(out), f64(logits)
        assert (got[:, :, V:] == (9 if place == "new" else x[:, :, V:])).all()
        for b in range(B):
            bias = np.zeros(V)
            for t, v in zip(ids[b], vals[b]):
                if 0 <= t < V:
                    bias[t] += np.float64(v)
            for i in range(R):
                if i > n[b]:
                    np.testing.assert_array_equal(got[b, i, :V], x[b, i, :V])
                    continue
                path = toks[b][[j - 1 for j in range(1, n[b] + 1) if (bits[b, i, j] if use_mask else j <= i)]]
                seen = np.concatenate([hist[b], path]).astype(np.int64)
                c = np.bincount(seen[(seen >= 0) & (seen < V)], minlength=V).astype(np.float64)
                with np.errstate(invalid="ignore"):
                    want, size = E.adjust(x[b, i, :V], V, c, f64(rep)[b], f64(pres)[b], f64(freq)[b], bias,
                                          allowed[b, i] if use_allowed else None)
                y = got[b, i, :V]
                fin = np.isfinite(want)
                np.testing.assert_array_equal(y[~fin], want[~fin])
                tol = 6 * U * size[fin] + (2.0 ** -8 * np.abs(want[fin]) if dtype == "bf16" else 0)
                assert (np.abs(y[fin] - want[fin]) <= tol).all()


def test_adjust_logits_bad_penalty_leaves_rows_alone(ver):
    x = torch.randn(3, 2, 64, device=DEV)
    y = torch.zeros_like(x)
    ver.adjust_logits(x, out=y, history=ints([[1, 2]] * 3), tokens=ints([[3]] * 3),
                      rep_penalty=torch.tensor([1.5, 0.0, float("nan")], device=DEV))
    assert ver.error() == binding.SV_ERR_STATE
    assert torch.equal(y[1:], x[1:]) and not torch.equal(y[0], x[0])


# --------------------------------------------------------------------------- #
# refusals: nothing is launched
# --------------------------------------------------------------------------- #
def test_refusals(ver):
    bf = dict(dtype=torch.bfloat16, device=DEV)
    q, kv, t, S = torch.zeros(1, 2, 4, 64, **bf), torch.zeros(2, 1, 2, 2, 16, 64, **bf), ints([[0]]), ints([0])

    def refused(fn, code=None):
        with pytest.raises(binding.SvError if code else ValueError) as e:
            fn()
        assert code is None or e.value.code == code

    INV, UNS = binding.SV_ERR_INVALID, binding.SV_ERR_UNSUPPORTED
    refused(lambda: ver.tree_attention(q[:, :, :3], kv, t, S), INV)                       # 3 heads over 2
    refused(lambda: ver.tree_attention(q.float(), kv, t, S), UNS)                          # fp32 over bf16
    refused(lambda: ver.tree_attention(q, kv, t, S, layer=1), INV)
    refused(lambda: ver.tree_attention(q, kv, t, S, scale=float("nan")), INV)
    refused(lambda: ver.tree_attention(q, kv, t, S, stage=torch.zeros(1, 1, 1, 2, 2, 64, **bf)), INV)  # 1 row of 2
    refused(lambda: ver.tree_attention(q, kv, t, S, stage=torch.zeros(1, 2, 1, 2, 2, 64, device=DEV)), INV)
    refused(lambda: ver.tree_attention(torch.zeros(1, 2, 4, 72, **bf)[..., 8:], kv, t, S, out=torch.zeros_like(q)[..., :63]))
    refused(lambda: ver.tree_attention(torch.zeros(1, 2, 4, 68, **bf)[..., 4:], kv, t, S), INV)         # unaligned
    refused(lambda: ver.tree_attention(q, kv.cpu(), t, S))
    refused(lambda: ver.tree_attention(q, kv, t.long(), S))
    refused(lambda: ver.tree_attention(q, kv, t, S, n_nodes=ints([])))
    a = binding.make_attention_args(q, kv, t, S, torch.empty_like(q))
    ws = torch.zeros(binding.sv_attention_workspace_size(ver.handle, a), dtype=torch.uint8, device=DEV)
    refused(lambda: binding.sv_tree_attention(ver.handle, a, ws[:-256]), INV)
    refused(lambda: binding.sv_tree_attention(None, a, ws), INV)
    k = torch.zeros(1, 2, 2, 64, **bf)
    refused(lambda: ver.kv_append(k, k, S))
    refused(lambda: ver.kv_append(k, k, S, kv=kv))
    refused(lambda: ver.kv_append(k, k.float(), S, kv=kv, block_table=t))
    refused(lambda: ver.kv_append(k, k, S, kv=kv, block_table=t, rope=torch.zeros(4, 33, 2, device=DEV)), INV)
    refused(lambda: ver.kv_append(k, k, S, stage=torch.zeros(1, 1, 1, 2, 2, 64, **bf)), INV)
    refused(lambda: ver.kv_read(torch.zeros(1, 2, 2, 2, 32, **bf), S, kv=kv, block_table=t))
    refused(lambda: ver.kv_read(torch.zeros(1, 2, 2, 2, 64, dtype=torch.float16, device=DEV), S, kv=kv, block_table=t))
    refused(lambda: ver.tree_mask(torch.zeros(1, binding.SV_TREE_MAX_NODES + 1, dtype=torch.int32, device=DEV)), INV)
    refused(lambda: ver.tree_mask(torch.zeros(1, 40, dtype=torch.int32, device=DEV),
                                  out=dict(mask=ints(np.zeros((1, 41, 1))), depth=ints(np.zeros((1, 41))))), INV)
    x = torch.zeros(1, 2, 64, **bf)
    refused(lambda: ver.adjust_logits(x), INV)                                             # two rows, no tokens
    refused(lambda: ver.adjust_logits(x, V=65, tokens=ints([[1]])), INV)
    refused(lambda: ver.adjust_logits(x, tokens=ints([[1]]), allowed=ints(np.zeros((1, 2, 1)))), INV)
    refused(lambda: ver.adjust_logits(x, tokens=ints([[1]]), bias_ids=ints([[1, 2]]),
                                      bias_values=torch.zeros(1, 3, device=DEV)))
    refused(lambda: ver.adjust_logits(torch.zeros(1, 2, 60, **bf), tokens=ints([[1]])), INV)  # 120-byte rows
    torch.cuda.synchronize()
    assert ver.error() == 0


def test_empty_batches(ver):
    e = torch.zeros(0, 3, 4, 64, dtype=torch.bfloat16, device=DEV)
    kv = torch.zeros(2, 1, 2, 4, 16, 64, dtype=torch.bfloat16, device=DEV)
    t, S = torch.zeros(0, 2, dtype=torch.int32, device=DEV), ints([])
    assert ver.tree_attention(e, kv, t, S).shape == e.shape
    ver.kv_append(e, e, S, kv=kv, block_table=t)
    ver.tree_mask(torch.zeros(0, 3, dtype=torch.int32, device=DEV))
    ver.adjust_logits(torch.zeros(0, 1, 64, device=DEV))
    assert ver.error() == 0
