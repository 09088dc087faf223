"""Attention where a row's largest score moves along the keys, within tiles and
between them, so that weights and outputs are rescaled on the way; against the
fp64 definition.

Bounds, derived before any run: weights rounded to 8 bits, 2^-8, the fp32 terms
below 2^-10 (scores' sizes stay under 40: 2 (D + 3) 2^-24 40 < 2^-10), in units of
sum p |v|, and the output's own 2^-8 |o|.
"""

import os

import numpy as np
import pytest
import torch

from oracle import entries as E
from speculative_decoding_verification_07_gb300 import binding

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


def course(name, n, rng):
    """Scores' course over n keys, 0 .. 1."""
    x = np.arange(n) / n
    return {"rising": x, "falling": 1 - x, "waves": 0.5 - 0.5 * np.cos(x * 40), "late": (x > 0.9) * 1.0,
            "steps": np.floor(x * 7) / 7, "spikes": (rng.random(n) < 0.01) * 1.0}[name]


# rows of a head: 4 (a tile holds them four times), 45 (twice), 100, 250 (two tiles)
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("D,Hq,H,n,S", [(128, 8, 2, 0, 1000), (64, 8, 2, 0, 700), (128, 6, 2, 14, 611),
                                        (64, 4, 1, 24, 300), (128, 10, 1, 24, 900), (64, 6, 2, 32, 517)])
@pytest.mark.parametrize("name", ["rising", "falling", "waves", "late", "steps", "spikes"])
def test_moving_maximum(ver, name, fmt, D, Hq, H, n, S):
    rng = np.random.default_rng(len(name) + D + S)
    BS, N = 16, S + n + 1
    u = rng.choice([-1.0, 1.0], (H, D))
    k = course(name, N, rng)[:, None, None] * u * (30 / D ** 0.5) + 0.1 * rng.standard_normal((N, H, D))
    v = rng.standard_normal((N, H, D))
    q = np.repeat(u, Hq // H, 0) * rng.choice([-1.0, 0.5, 1.0], (n + 1, Hq, 1))  # falling, half as steep, rising
    k, v, q = (torch.tensor(x, dtype=torch.bfloat16, device=DEV)[None] for x in (k, v, q))
    blocks = -(-N // BS)
    row = D + E.TAIL if fmt == "e4m3" else D
    kv = torch.zeros(blocks, 1, 2, H, BS, row, dtype=torch.uint8 if fmt == "e4m3" else torch.bfloat16, device=DEV)
    table = torch.tensor(rng.permutation(blocks)[None], dtype=torch.int32, device=DEV)
    zero = torch.zeros(1, dtype=torch.int32, device=DEV)
    ver.kv_append(k, v, zero, kv=kv, block_table=table)
    held = ver.kv_read(torch.empty(1, N, 2, H, D, device=DEV), zero, kv=kv, block_table=table)[0].double().cpu().numpy()
    got = ver.tree_attention(q, kv, table, zero + S)[0].double().cpu().numpy()
    assert ver.error() == 0
    qd = q[0].double().cpu().numpy()
    for i in range(n + 1):
        seen = np.arange(N) <= S + i
        for h in range(Hq):
            o, size, scores = E.attend(qd[i, h], held[:, 0, h * H // Hq], held[:, 1, h * H // Hq], seen, D ** -0.5)
            assert scores < 40
            d = np.abs(got[i, h] - o)
            assert (d <= (2.0 ** -8 + 2.0 ** -10) * size + 2.0 ** -8 * np.abs(o)).all(), (i, h, d.max())


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_hidden_entries_of_tiny_scores(ver, fmt):
    """Scores that underflow are 0, and entries that a row does not see stay out
    all the same: the row is the mean of what it sees."""
    B, R, H, D, BS = 1, 6, 2, 128, 16
    g = torch.Generator(DEV).manual_seed(1)
    k = (torch.randn(B, R, H, D, generator=g, device=DEV) * 2.0 ** -118).bfloat16()
    q = (torch.randn(B, R, 8, D, generator=g, device=DEV) * 2.0 ** -118).bfloat16()
    v = torch.randn(B, R, H, D, generator=g, device=DEV).bfloat16()
    row = D + E.TAIL if fmt == "e4m3" else D
    kv = torch.zeros(1, 1, 2, H, BS, row, dtype=torch.uint8 if fmt == "e4m3" else torch.bfloat16, device=DEV)
    zero = torch.zeros(1, dtype=torch.int32, device=DEV)
    table = torch.zeros(1, 1, dtype=torch.int32, device=DEV)
    ver.kv_append(k, v, zero, kv=kv, block_table=table)
    held = ver.kv_read(torch.empty(B, R, 2, H, D, device=DEV), zero, kv=kv, block_table=table)[0, :, 1].double()
    got = ver.tree_attention(q, kv, table, zero)[0].double()
    assert ver.error() == 0
    for i in range(R):
        o = held[:i + 1].mean(0).repeat_interleave(4, 0)
        size = held[:i + 1].abs().mean(0).repeat_interleave(4, 0)
        assert ((got[i] - o).abs() <= (2.0 ** -8 + 2.0 ** -10) * size + 2.0 ** -8 * o.abs()).all()
