"""Forms of the scores where the factors that make a score are near the ends of fp32: queries of
2^-119 on keys of 2^117 and the other way round, the smallest caps, rows and keys that score 0
beside them.

Bounds: those of test_gpu_attention_forms, where a factor of the scores may be subnormal with 19
bits (2^-19 of a score's size more; scores are below 40, so 2 x 40 x 2^-19 < 2^-12 of sum p |v|)."""

import os

import numpy as np
import pytest
import torch

from oracle import entries as E
from speculative_decoding_verification_07_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24


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


TYPES = {"bf16": torch.bfloat16, "e4m3": torch.uint8, "fp32": torch.float32}


def cache(ver, fmt, k, v):
    """k, v [n, D]: a cache that holds them (position i at block and slot of a shuffled table), and
    what it holds in fp64."""
    n, D = k.shape
    dt = torch.float32 if fmt == "fp32" else torch.bfloat16
    k, v = (torch.tensor(x, dtype=dt, device=DEV) for x in (k, v))
    row = D + E.TAIL if fmt == "e4m3" else D
    kv = torch.zeros(-(-n // 16), 1, 2, 1, 16, row, dtype=TYPES[fmt], device=DEV)
    t = torch.randperm(len(kv), generator=torch.Generator().manual_seed(n)).int()[None].to(DEV)
    for at in range(0, n, 64):
        ver.kv_append(k[None, at:at + 64, None], v[None, at:at + 64, None], ints([at]), kv=kv, block_table=t)
    held = ver.kv_read(torch.empty(1, n, 2, 1, D, device=DEV), ints([0]), kv=kv, block_table=t)[0, :, :, 0]
    return kv, t, held.double().cpu().numpy()


def check(ver, fmt, kv, t, held, q, scale=None, most=40, **form):
    """One entry's G heads over all n positions against the definition."""
    (G, D), n = q.shape, held.shape[0]
    q = torch.tensor(q, dtype=torch.float32 if fmt == "fp32" else torch.bfloat16, device=DEV)
    sc = D ** -0.5 if scale is None else scale
    call = dict(form)
    if "slopes" in form:
        call["slopes"] = torch.tensor(form["slopes"], device=DEV)
    got = ver.tree_attention(q[None, None], kv, t, ints([n - 1]), scale=scale, **call)[0, 0].double().cpu().numpy()
    assert ver.error() == 0
    far, qd = np.arange(n - 1, -1, -1), q.double().cpu().numpy()
    for h in range(G):
        slope = float(form["slopes"][h]) if "slopes" in form else None
        o, size, scores, drop = E.attend_shaped(qd[h], held[:, 0], held[:, 1], np.ones(n, bool), sc, far, form.get("softcap"), slope,
                                                form.get("window"))
        assert scores < most
        scores = 2 * ((D + 11) * U * min(scores, 40) + 2 * U * drop) + 2.0 ** -12
        tol = (scores + 2 * (n + 16) * U) * size if fmt == "fp32" else (2.0 ** -8 + 2.0 ** -10 + scores) * size + 2.0 ** -8 * np.abs(o)
        assert (np.abs(got[h] - o) <= tol).all(), (h, np.abs(got[h] - o).max(), got[h][:4], o[:4])


def forms(G):
    slopes = np.float32(2.0) ** (-8 * np.arange(1, G + 1, dtype=np.float32) / G)
    return {"cap": dict(softcap=5.0), "wide cap": dict(softcap=400.0), "slopes": dict(slopes=slopes), "window": dict(window=10 ** 6),
            "both": dict(softcap=20.0, slopes=slopes), "all": dict(softcap=100.0, slopes=slopes, window=45)}


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "fp32"])
@pytest.mark.parametrize("G", [4, 40, 150])
@pytest.mark.parametrize("form", list(forms(1)))
@pytest.mark.parametrize("e", [-117, 0, 100])
def test_tiny_queries_and_huge_keys(ver, fmt, G, form, e):
    """Ordinary scores of factors of 2^e and 2^-e."""
    rng = np.random.default_rng(G)
    k, v = 2.0 ** -e * rng.standard_normal((50, 128)), rng.standard_normal((50, 128))
    check(ver, fmt, *cache(ver, fmt, k, v), 2.0 ** e * rng.choice([-0.25, 0.25], (G, 128)), **forms(G)[form])


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "fp32"])
@pytest.mark.parametrize("G", [3, 40, 150])
@pytest.mark.parametrize("cap", [2.0 ** -60, 2.0 ** -20, 1.0])
def test_smallest_caps_under_large_queries(ver, fmt, G, cap):
    """Scores of 0, exactly, beside scores far past the cap: keys that a query's two halves cancel on,
    and queries of zeros.  (Products of 2^90 and the factor of the smallest cap, 2^60, are no fp32 value.)"""
    rng = np.random.default_rng(G)
    k = rng.choice([-1.0, 1.0], (40, 128))
    k[::3, 64:] = k[::3, :64]
    half = 2.0 ** 90 * rng.choice([0.5, 1.0], (G, 64))
    q = np.concatenate([half, -half], 1)
    q[1] = 0
    check(ver, fmt, *cache(ver, fmt, k, rng.standard_normal((40, 128))), q, scale=0.125, softcap=cap, most=np.inf)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "fp32"])
@pytest.mark.parametrize("e", [-100, 80])
@pytest.mark.parametrize("cap", [2.0 ** -60, 30.0])
def test_scales_of_any_size(ver, fmt, e, cap):
    """The scale makes up for keys of 2^-e; a query of zeros weighs all keys the same."""
    rng = np.random.default_rng(3)
    k, q = 2.0 ** -e * rng.standard_normal((50, 128)), rng.choice([-0.25, 0.25], (5, 128))
    q[2] = 0
    held = cache(ver, fmt, k, rng.standard_normal((50, 128)))
    check(ver, fmt, *held, q, scale=2.0 ** (e - 3), softcap=cap)
    if cap == 30.0:
        check(ver, fmt, *held, q, scale=2.0 ** (e - 3), slopes=np.float32([0.0, 0.5, 0.01, -0.1, 0.001]))


@pytest.mark.parametrize("fmt,D", [("fp32", 128), ("fp32", 64), ("bf16", 80), ("e4m3", 96)])
@pytest.mark.parametrize("form", list(forms(1)))
def test_products_past_fp32_under_a_small_scale(ver, fmt, D, form):
    """Heads that are multiplied in fp32: the scale comes before the product, as without a form."""
    rng = np.random.default_rng(D)
    k, q = 2.0 ** 64 * rng.standard_normal((50, D)), 2.0 ** 64 * rng.choice([-0.25, 0.25], (6, D))
    check(ver, fmt, *cache(ver, fmt, k, rng.standard_normal((50, D))), q, scale=2.0 ** -128, **forms(6)[form])
