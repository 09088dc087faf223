"""Infinities, NaN and zeros where entries are rotated, decoded and attended."""

import os

import numpy as np
import pytest
import torch

from oracle import entries as E
from speculative_decoding_verification_07_gb300 import binding, rope

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


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


@pytest.mark.parametrize("G", [4, 40, 150])
def test_a_scale_of_zero_is_zero(ver, G):
    """value = code * scale: keys of scale 0 score 0 whatever their codes, values
    of scale 0 are 0.  Held to the bound of the attention's own tests."""
    D, n = 128, 50
    rng = np.random.default_rng(G)
    g = torch.Generator(DEV).manual_seed(G)
    k, v = torch.randn(2, 1, n, 1, D, generator=g, device=DEV).bfloat16()
    kv = torch.zeros(4, 1, 2, 1, 16, D + E.TAIL, dtype=torch.uint8, device=DEV)
    t = ints([[3, 0, 1, 2]])
    ver.kv_append(k, v, ints([0]), kv=kv, block_table=t)
    for which, i in ((0, 3), (0, 40), (1, 7), (1, 33)):
        kv[t[0, i // 16], 0, which, 0, i % 16, D:] = 0
    held = ver.kv_read(torch.empty(1, n, 2, 1, D, device=DEV), ints([0]), kv=kv, block_table=t)[0, :, :, 0].double().cpu().numpy()
    assert not held[[3, 40], 0].any() and not held[[7, 33], 1].any()
    q = torch.tensor(rng.standard_normal((G, D)) * 3, dtype=torch.bfloat16, device=DEV)
    got = ver.tree_attention(q[None, None], kv, t, ints([n - 1]))[0, 0].double().cpu().numpy()
    assert ver.error() == 0
    for h in range(G):
        o, size, _ = E.attend(q[h].double().cpu().numpy(), held[:, 0], held[:, 1], np.ones(n, bool), D ** -0.5)
        assert (np.abs(got[h] - o) <= (2.0 ** -8 + 2.0 ** -10) * size + 2.0 ** -8 * np.abs(o)).all()


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("G", [4, 40, 150])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_a_query_that_is_not_finite_gives_nan(ver, fmt, G, bad):
    """Its scores are infinite or NaN, with one infinity of each sign among them."""
    D, n, H = 128, 40, 1
    g = torch.Generator(DEV).manual_seed(G)
    k = torch.randn(1, n, H, D, generator=g, device=DEV).bfloat16()
    k[..., 5] *= 2.0 ** -12  # codes of 2^-3 and less: half of the largest number times them is finite
    row = D + E.TAIL if fmt == "e4m3" else D
    kv = torch.zeros(3, 1, 2, H, 16, row, dtype=torch.uint8 if fmt == "e4m3" else torch.bfloat16, device=DEV)
    t = ints([[2, 0, 1]])
    ver.kv_append(k, k, ints([0]), kv=kv, block_table=t)
    q = torch.randn(1, 1, G, D, generator=g, device=DEV).bfloat16()
    want = ver.tree_attention(q, kv, t, ints([n - 1]))
    q[0, 0, 2, 5] = bad
    got = ver.tree_attention(q, kv, t, ints([n - 1]))
    assert ver.error() == 0
    assert torch.isnan(got[0, 0, 2]).all()
    others = [h for h in range(G) if h != 2]
    assert torch.equal(got[0, 0, others], want[0, 0, others])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rot,pairs", [(16, False), (16, True), (6, False), (6, True), (12, True)])
def test_columns_past_the_rotation_pass_unchanged(ver, dtype, rot, pairs):
    """Bit for bit, whatever they and their neighbours hold (a NaN: any NaN)."""
    D, R, H = 64, 5, 2
    g = torch.Generator(DEV).manual_seed(rot)
    x = torch.randn(1, R, H, D, generator=g, device=DEV).to(dtype)
    special = torch.tensor([float("inf"), -float("inf"), float("nan"), -0.0, 0.0, 3.0, 1e-39, float("inf")], dtype=dtype, device=DEV)
    x[:, 1:, :, rot:] = special.repeat(D)[:D - rot]
    x[:, 2:, :, rot:] = special.repeat(D)[1:D - rot + 1]
    stage = torch.zeros(1, R, 1, 2, H, D, dtype=dtype, device=DEV)
    q = ver.kv_append(x, x, ints([3]), q=x, stage=stage, interleaved=pairs, rope=rope.rope_table(16, rope.rope_frequencies(rot)))
    assert ver.error() == 0
    word = torch.int16 if dtype == torch.bfloat16 else torch.int32
    for y in (q, stage[:, :, 0, 0]):
        got, want = y[..., rot:].contiguous(), x[..., rot:].contiguous()
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(got.view(word)[~torch.isnan(got)], want.view(word)[~torch.isnan(want)])
        assert torch.isfinite(y[..., :rot]).all()
        assert not torch.equal(y[..., :rot], x[..., :rot])


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("G", [4, 40, 150])
def test_tiny_queries_and_huge_keys(ver, fmt, G):
    """Ordinary scores of factors near both ends of fp32 (a factor of the scores may be
    subnormal, with 20 bits: 2^-20 of a score's size more), held to the bound of
    the attention's own tests."""
    D, n = 128, 50
    rng = np.random.default_rng(G)
    bf = lambda x: torch.tensor(x, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    k, v = bf(2.0 ** 117 * rng.standard_normal((n, D))), bf(rng.standard_normal((n, D)))
    row = D + E.TAIL if fmt == "e4m3" else D
    kv = torch.zeros(4, 1, 2, 1, 16, row, dtype=torch.uint8 if fmt == "e4m3" else torch.bfloat16, device=DEV)
    t = ints([[3, 0, 1, 2]])
    ver.kv_append(k[None, :, None], v[None, :, None], ints([0]), kv=kv, block_table=t)
    held = ver.kv_read(torch.empty(1, n, 2, 1, D, device=DEV), ints([0]), kv=kv, block_table=t)[0, :, :, 0].double().cpu().numpy()
    q = bf(2.0 ** -117 * rng.choice([-0.25, 0.25], (G, D)))
    got = ver.tree_attention(q[None, None], kv, t, ints([n - 1]))[0, 0].double().cpu().numpy()
    assert ver.error() == 0
    for h in range(G):
        o, size, scores = E.attend(q[h].double().cpu().numpy(), held[:, 0], held[:, 1], np.ones(n, bool), D ** -0.5)
        assert 1 < scores < 40
        assert (np.abs(got[h] - o) <= (2.0 ** -8 + 2.0 ** -10) * size + 2.0 ** -8 * np.abs(o)).all()
