"""Types and shapes that the calls around the verification step refuse, since they
would be read as others."""

import os

import numpy as np
import pytest
import torch

from speculative_decoding_verification_07_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
I32, F32 = torch.int32, torch.float32


@pytest.fixture(scope="module")
def ver():
    if not os.path.exists(binding.LIB_PATH):
        from speculative_decoding_verification_07_gb300 import build
        build.build()
    v = binding.Verifier(0)
    yield v
    v.close()


def zeros(*shape, dtype=I32):
    return torch.zeros(*shape, dtype=dtype, device=DEV)


def calls(ver, changed):
    """One valid call of each operator with one argument of another type or shape."""
    B, R, N, H, D = 2, 3, 2, 2, 64
    k, kv, table = zeros(B, R, H, D, dtype=F32), zeros(4, 1, 2, H, 16, D, dtype=F32), ints([[0, 1], [2, 3]])
    a = dict(seq_len=zeros(B), n_nodes=zeros(B), depth=zeros(B, R), mask=zeros(B, R, 1), parent=zeros(B, N),
             history=zeros(B, 5), tokens=zeros(B, N), rep_penalty=zeros(B, dtype=F32) + 1, presence=zeros(B, dtype=F32),
             frequency=zeros(B, dtype=F32), bias_ids=zeros(B, 3), bias_values=zeros(B, 3, dtype=F32),
             allowed=zeros(B, R, 1), mask_out=zeros(B, R, 1), depth_out=zeros(B, R), table=table)
    a.update(changed)
    ver.tree_mask(a["parent"], n_nodes=a["n_nodes"], out=dict(mask=a["mask_out"], depth=a["depth_out"]))
    ver.kv_append(k, k, a["seq_len"], kv=kv, block_table=a["table"], depth=a["depth"], n_nodes=a["n_nodes"])
    ver.kv_read(zeros(B, R, 2, H, D, dtype=F32), a["seq_len"], kv=kv, block_table=a["table"], n_nodes=a["n_nodes"])
    ver.tree_attention(k, kv, a["table"], a["seq_len"], n_nodes=a["n_nodes"], mask=a["mask"])
    ver.adjust_logits(zeros(B, R, 32, dtype=F32), mask=a["mask"], n_nodes=a["n_nodes"],
                      **{x: a[x] for x in ("history", "tokens", "rep_penalty", "presence", "frequency", "bias_ids",
                                           "bias_values", "allowed")})


def ints(x):
    return torch.tensor(x, dtype=I32, device=DEV)


def other(shape, dtype):
    return zeros(*shape).view(dtype) if dtype == torch.uint32 else zeros(*shape, dtype=dtype)


def test_the_valid_calls(ver):
    calls(ver, {})
    calls(ver, dict(mask=zeros(2, 3, 1).view(torch.uint32), allowed=zeros(2, 3, 1).view(torch.uint32)))  # words
    torch.cuda.synchronize()
    assert ver.error() == 0


@pytest.mark.parametrize("name,shape", [("seq_len", (2,)), ("n_nodes", (2,)), ("depth", (2, 3)), ("mask", (2, 3, 1)),
                                        ("history", (2, 5)), ("tokens", (2, 2)), ("bias_ids", (2, 3)), ("allowed", (2, 3, 1)),
                                        ("mask_out", (2, 3, 1)), ("depth_out", (2, 3)), ("parent", (2, 2)), ("table", (2, 2))])
def test_whole_numbers_are_int32(ver, name, shape):
    for dtype in (F32, torch.int64) + (() if name in ("mask", "allowed", "mask_out") else (torch.uint32,)):
        with pytest.raises(ValueError):
            calls(ver, {name: other(shape, dtype)})


@pytest.mark.parametrize("name,shape", [("rep_penalty", (2,)), ("presence", (2,)), ("frequency", (2,)), ("bias_values", (2, 3))])
def test_factors_are_fp32(ver, name, shape):
    for dtype in (I32, torch.uint32, torch.float64, torch.bfloat16):
        with pytest.raises(ValueError):
            calls(ver, {name: other(shape, dtype)})


def test_tables_of_another_width_are_refused(ver):
    """Padded draft buffers would be read as rows of R - 1 (or R) values."""
    B, R, D = 2, 4, 64
    x = torch.zeros(B, R, 64, device=DEV)
    k = torch.zeros(B, R, 1, D, device=DEV)
    stage = torch.zeros(B, R, 1, 2, 1, D, device=DEV)
    zero = torch.zeros(B, dtype=torch.int32, device=DEV)
    for w in (R - 2, R, R + 5):
        with pytest.raises(ValueError):
            ver.adjust_logits(x, tokens=torch.zeros(B, w, dtype=torch.int32, device=DEV))
    with pytest.raises(ValueError):
        ver.adjust_logits(x, tokens=torch.zeros(R - 1, B, dtype=torch.int32, device=DEV))
    ver.adjust_logits(x, tokens=torch.zeros(B, R - 1, dtype=torch.int32, device=DEV))
    for w in (R - 1, R + 1):
        with pytest.raises(ValueError):
            ver.kv_append(k, k, zero, stage=stage, depth=torch.zeros(B, w, dtype=torch.int32, device=DEV))
    ver.kv_append(k, k, zero, stage=stage, depth=torch.zeros(B, R, dtype=torch.int32, device=DEV))
    with pytest.raises(ValueError):  # depths of a mask call, where they are given
        ver.tree_mask(torch.zeros(2, B, dtype=torch.int32, device=DEV), out=dict(mask=torch.zeros(2, B + 1, 1, dtype=torch.int32, device=DEV),
                                                               depth=torch.zeros(2, B + 4, dtype=torch.int32, device=DEV)))
    torch.cuda.synchronize()
    assert ver.error() == 0
