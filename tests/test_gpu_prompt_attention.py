"""Attention of prompts and of other passes with more rows than a CTA holds: many
row blocks a head, ragged, with and without a mask; against the fp64 definition,
at the bounds of the attention's other tests."""

import os

import numpy as np
import pytest

from speculative_decoding_verification_07_gb300 import binding
from tests.test_gpu_entries import check_attention, tree_bits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ver():
    if not os.path.exists(binding.LIB_PATH):
        from speculative_decoding_verification_07_gb300 import build
        build.build()
    v = binding.Verifier(0)
    yield v
    v.close()


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "fp32"])
@pytest.mark.parametrize("staged,mask", [(False, False), (True, False), (False, True), (True, True)])
def test_prompts(ver, fmt, staged, mask):
    """257 positions of 3 heads a group (771 rows in four blocks), a part of them, one, none."""
    R = 257
    bits = np.repeat(np.tril(np.ones((R, R), bool))[None], 4, 0)
    check_attention(ver, fmt, 128, 6, 2, [0, 131, 40, 7], [R - 1, 128, 0, -1], bits, staged, seed=21, mask=mask)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("D,Hq,H", [(128, 7, 1), (64, 7, 1)])
def test_requests_of_one_and_two_row_tiles(ver, fmt, D, Hq, H):
    """28, 140, 315 and 427 rows a head in one call."""
    check_attention(ver, fmt, D, Hq, H, [700, 129, 300, 5], [3, 19, 44, 60], tree_bits("random:60", 4, 60), True, seed=22)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_more_requests_than_threads(ver, fmt):
    """Each thread of a CTA walks several requests."""
    rng = np.random.default_rng(23)
    B = 900
    check_attention(ver, fmt, 64, 2, 1, rng.integers(0, 40, B), rng.integers(-1, 2, B), tree_bits("chain:1", B, 1), True, seed=24)
