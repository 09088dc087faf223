"""Pins of oracle/entries.py on facts outside it, and CPU checks of the rotary
tables and of the binding's argument checks."""

import math

import numpy as np
import pytest
import torch

from oracle import entries as E
from speculative_decoding_verification_07_gb300 import binding, rope


def test_ancestors_of_a_hand_drawn_tree():
    #   0 -> 1, 2;  1 -> 3;  2 -> 4;  4 -> 5
    bits, depth = E.ancestors([0, 0, 1, 2, 4], 5)
    assert [set(np.flatnonzero(r)) for r in bits] == [{0}, {0, 1}, {0, 2}, {0, 1, 3}, {0, 2, 4}, {0, 2, 4, 5}]
    assert depth.tolist() == [0, 1, 1, 2, 2, 3]
    bits, depth = E.ancestors([0, 0, 1, 2, 4], 2)
    assert not bits[3:].any() and not depth[3:].any()
    assert E.pack(np.eye(33, dtype=bool))[32].tolist() == [0, 1]


def test_e4m3_values_and_rounding_are_the_formats():
    codes = np.arange(256)
    ref = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(E.e4m3_value(codes), ref)
    x = np.concatenate([np.linspace(-448, 448, 20001), np.linspace(-0.02, 0.02, 4001), [2.0 ** -10, 3 * 2.0 ** -10]])
    ref = torch.tensor(x).to(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(E.e4m3_round(x), ref)


def test_e4m3_scale_is_the_smallest_that_fits():
    x = np.abs(np.random.default_rng(0).standard_normal((500, 3))) * 10.0 ** np.arange(-20, 10, 0.06)[:, None]
    s = E.e4m3_scale(x)
    assert (x.max(-1) <= 448 * s).all() and (x.max(-1) > 224 * s).all()
    assert E.e4m3_scale(np.zeros((1, 4)))[0] == 1 and E.e4m3_scale(np.array([[448.0]]))[0] == 1


@pytest.mark.parametrize("pairs", [False, True])
def test_rotation_keeps_norms_and_depends_on_the_distance(pairs):
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((2, 16))
    f = rope.rope_frequencies(12).numpy()
    rot = lambda x, p: E.rotate(x, np.cos(p * f), np.sin(p * f), pairs)  # noqa: E731
    assert np.allclose(np.linalg.norm(rot(q, 77)), np.linalg.norm(q))
    assert np.allclose(rot(q, 9) @ rot(k, 4), rot(q, 105) @ rot(k, 100))
    assert (rot(q, 5)[12:] == q[12:]).all()


def test_attend_is_the_mean_under_equal_scores_and_zero_without_keys():
    V = np.arange(12.0).reshape(4, 3)
    o, _, _ = E.attend(np.zeros(3), np.ones((4, 3)), V, np.array([1, 0, 1, 1], bool), 1.0)
    assert np.allclose(o, V[[0, 2, 3]].mean(0))
    assert not E.attend(np.zeros(3), np.ones((4, 3)), V, np.zeros(4, bool), 1.0)[0].any()


def test_adjust_by_hand():
    l, _ = E.adjust(np.array([2.0, -2.0, 1.0, 5.0]), 4, np.array([2, 1, 0, 0]), 2.0, 0.25, 0.5,
                    np.array([0, 0, 3.0, 0]), np.array([True, True, True, False]))
    assert l.tolist() == [1 - 1.25, -4 - 0.75, 4.0, -math.inf]


def test_rope_frequency_rules():
    f = rope.rope_frequencies(64)
    assert f[0] == 1 and torch.allclose(f[16], torch.tensor(10000.0 ** -0.5, dtype=torch.float64))
    assert torch.allclose(rope.rope_frequencies(64, scaling="linear", factor=4.0), f / 4)
    g = rope.rope_frequencies(64, scaling="base", factor=8.0)
    assert g[0] == 1 and torch.allclose(g[-1], f[-1] / 8)
    h = rope.rope_frequencies(64, scaling="bands", factor=8.0, original=4096)
    turns = 4096 * f / (2 * math.pi)
    assert torch.equal(h[turns > 32], f[turns > 32]) and torch.allclose(h[turns < 1], f[turns < 1] / 8)
    assert ((h <= f) & (h >= f / 8 - 1e-18)).all() and (h.diff() < 0).all()
    t = rope.rope_table(100000, f, attention_factor=1.5, device="cpu")
    assert t.shape == (100000, 32, 2) and t.dtype == torch.float32
    assert abs(t[99999, 3, 1].item() - 1.5 * math.sin(99999 * f[3].item())) < 1e-6
    for kw in (dict(scaling="other"), dict(scaling="bands")):
        with pytest.raises(ValueError):
            rope.rope_frequencies(64, **kw)
    with pytest.raises(ValueError):
        rope.rope_frequencies(7)


def test_payload_of_an_eight_bit_cache_moves_two_byte_elements(monkeypatch):
    monkeypatch.setattr(binding, "_ptr", lambda t: 0)
    p = binding._payload(torch.zeros(2, 3, 2, 4, 16, 128 + 16, dtype=torch.uint8))
    assert (p.layers, p.heads, p.head_dim, p.elem_bytes) == (3, 4, 72, 2)
