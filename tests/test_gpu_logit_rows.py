"""Rows of the logit rules at the edges of their layouts."""

import os

import pytest
import torch

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


@pytest.mark.parametrize("masked", [False, True])
def test_more_than_65536_drafted_tokens(ver, masked):
    """A node counts from its own row on, whatever its number."""
    V, R, node = 8, 66000, 65536 + 40
    x = torch.ones(1, R, V, device=DEV)
    tokens = torch.full((1, R - 1), -1, dtype=torch.int32, device=DEV)  # ids outside [0, V) are ignored
    tokens[0, node - 1] = 3
    tokens[0, 100 - 1] = 3
    tokens[0, node + 50 - 1] = 5
    kw = {}
    if masked:  # every node sees itself alone but for one row, which sees the late node
        mask = torch.zeros(1, R, (R + 31) // 32, dtype=torch.int32, device=DEV)
        mask[0, 7, node // 32] = 1 << node % 32
        mask[0, 9, (node - 65536) // 32] = 1 << node % 32
        kw["mask"] = mask
    y = ver.adjust_logits(x, out=torch.empty_like(x), tokens=tokens, frequency=torch.full((1,), 0.25, device=DEV), **kw)
    assert ver.error() == 0
    want = x.clone()
    if masked:
        want[0, 7, 3] -= 0.25
    else:
        want[0, 100:, 3] -= 0.25
        want[0, node:, 3] -= 0.25
        want[0, node + 50:, 5] -= 0.25
    assert torch.equal(y, want)


def test_more_rows_than_are_counted_are_refused(ver):
    R = (1 << 22) + 1
    with pytest.raises(binding.SvError) as e:
        ver.adjust_logits(torch.zeros(1, R, 4, device=DEV), tokens=torch.zeros(1, R - 1, dtype=torch.int32, device=DEV))
    assert e.value.code == binding.SV_ERR_UNSUPPORTED
    assert ver.error() == 0


def test_columns_past_a_view_are_refused(ver):
    """A view's rows may be followed by no more of their buffer."""
    whole = torch.zeros(1, 2, 128, device=DEV)
    tokens = torch.zeros(1, 1, dtype=torch.int32, device=DEV)
    view = whole[:, :, 64:]
    for x, out in ((view, whole), (whole, view)):
        with pytest.raises(binding.SvError) as e:
            ver.adjust_logits(x, out=out, V=65, tokens=tokens)
        assert e.value.code == binding.SV_ERR_INVALID
    ver.adjust_logits(view, V=64, tokens=tokens)
    torch.cuda.synchronize()
    assert ver.error() == 0


@pytest.mark.parametrize("B", [1, 3])
def test_one_row_a_request_out_of_longer_ones(ver, B):
    """One row of each request: the requests' distance is the row's stride."""
    V, T = 61, 4
    g = torch.Generator(DEV).manual_seed(B)
    rows = torch.randn(B, T, 64, generator=g, device=DEV)
    bias = dict(bias_ids=torch.full((B, 1), 60, dtype=torch.int32, device=DEV), bias_values=torch.ones(B, 1, device=DEV))
    for x in (rows[:, 2:3], rows[:, 3:, :V], rows[:, 1, :V].unsqueeze(1)):
        want = x[..., :V].clone()
        want[..., 60] += 1
        out = torch.empty(B, 1, 64, device=DEV)
        ver.adjust_logits(x, out=out, V=V, **bias)
        assert torch.equal(out[..., :V], want)
    keep = rows.clone()
    ver.adjust_logits(rows[:, 1, :V].unsqueeze(1), **bias)
    keep[:, 1, 60] += 1
    assert torch.equal(rows, keep)
    assert ver.error() == 0
