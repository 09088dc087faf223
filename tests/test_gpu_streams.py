"""The calls around the verification step on several streams: workspaces that grow
and outputs that are allocated while other streams are busy."""

import os

import pytest
import torch

from speculative_decoding_verification_07_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(binding.LIB_PATH):
        from speculative_decoding_verification_07_gb300 import build
        build.build()


@pytest.fixture
def ver():
    v = binding.Verifier(0)
    yield v
    torch.cuda.synchronize()
    v.close()


def job(B, S, R, seed, H=2, Hq=8, D=128, fmt=torch.bfloat16):
    """Inputs of an attention whose items are shared by CTAs (partial results)."""
    g = torch.Generator(DEV).manual_seed(seed)
    n = -(-(S + R) // 16)
    kv = torch.randn(B * n, 1, 2, H, 16, D, generator=g, device=DEV).to(fmt)
    t = torch.randperm(B * n, generator=g, device=DEV).int().reshape(B, n)
    q = torch.randn(B, R, Hq, D, generator=g, device=DEV).to(fmt)
    return q, kv, t, torch.full((B,), S, dtype=torch.int32, device=DEV)


def jobs():
    # growing workspaces: one row tile per CTA, then two, then the fp32 kernel's
    return [job(1, 700, 1, 1), job(1, 9000, 4, 2), job(2, 9000, 60, 3), job(4, 600, 3, 4, fmt=torch.float32, Hq=2)]


def test_a_workspace_that_grows_on_a_side_stream(ver):
    """The current stream allocates and fills blocks while the side stream's calls run."""
    work = jobs()
    alone = binding.Verifier(0)
    want = [alone.tree_attention(*j) for j in work]
    outs = [[torch.empty_like(w) for w in want] for _ in range(8)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    sizes = [w.numel() for w in alone._attention_workspaces.values()]
    for o in outs:
        for j, y in zip(work, o):
            ver.tree_attention(*j, out=y, stream=side)
            for n in sizes + [1 << 20, 1 << 22]:
                torch.full((n,), 255, dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    assert ver.error() == 0
    for o in outs:
        for y, w in zip(o, want):
            assert torch.equal(y, w)
    alone.close()


def test_calls_on_several_streams_at_once(ver):
    work = jobs()
    alone = binding.Verifier(0)
    want = [alone.tree_attention(*j) for j in work]
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [[torch.empty_like(w) for w in want] for _ in streams]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for rep in range(10):
        for x in range(len(work)):
            for i, s in enumerate(streams):
                at = (x + i) % len(work)  # other shapes beside one another
                if i == 0:
                    with torch.cuda.stream(s):
                        ver.tree_attention(*work[at], out=outs[i][at])
                else:
                    ver.tree_attention(*work[at], out=outs[i][at], stream=s)
    torch.cuda.synchronize()
    assert ver.error() == 0
    for o in outs:
        for y, w in zip(o, want):
            assert torch.equal(y, w)
    alone.close()


@pytest.mark.parametrize("warm", [False, True])
def test_a_captured_call_keeps_its_workspace(ver, warm):
    """A graph captured before the workspace grew is replayed after it; a call on
    the stream it was captured on does not wait for the graph's first run."""
    small, large = job(1, 9000, 4, 2), job(2, 9000, 60, 3)
    want = ver.tree_attention(*small)
    out, eager = torch.zeros_like(want), torch.zeros_like(want)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    if warm:
        ver.tree_attention(*small, out=out, stream=side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        ver.tree_attention(*small, out=out)
        ver.tree_attention(*small, out=out)
    ver.tree_attention(*small, out=eager, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(eager, want)
    ver.tree_attention(*large, out=torch.empty_like(large[0]), stream=side)
    keep = [torch.full((n,), 255, dtype=torch.uint8, device=DEV) for n in (1 << 22, 1 << 24, 5 << 22, 5 << 23) * 2]
    torch.cuda.synchronize()
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert all(k.eq(255).all() for k in keep)
    assert ver.error() == 0


@pytest.mark.parametrize("call", ["attention", "append", "mask"])
def test_outputs_allocated_for_another_stream(ver, call):
    """An output does not take memory that the current stream still reads."""
    side = torch.cuda.Stream()
    q, kv, t, S = job(2, 700, 8, 5)
    k = torch.randn(2, 8, 2, 128, device=DEV).bfloat16()
    stage = torch.zeros(2, 8, 1, 2, 2, 128, dtype=torch.bfloat16, device=DEV)
    parent = torch.zeros(2, 4095, dtype=torch.int32, device=DEV)
    run = {"attention": lambda **s: ver.tree_attention(q, kv, t, S, **s),
           "append": lambda **s: ver.kv_append(k, k, S, q=q, stage=stage, **s),
           "mask": lambda **s: ver.tree_mask(parent, **s)["mask"]}[call]
    torch.cuda.synchronize()
    want = run(stream=side)
    torch.cuda.synchronize()
    for _ in range(4):
        held = torch.full((want.untyped_storage().nbytes(),), 7, dtype=torch.uint8, device=DEV)
        copy = torch.zeros_like(held)
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)   # about 10 ms: the read below is still to come
        copy.copy_(held)
        del held                        # the current stream's to hand out again
        got = run(stream=side)
        torch.cuda.synchronize()
        assert copy.eq(7).all()
        assert torch.equal(got, want)
    # and, used on the current stream, it is not handed out on its own before that use
    got = run(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    copy = torch.empty_like(got)
    torch.cuda._sleep(20_000_000)
    copy.copy_(got)
    del got
    with torch.cuda.stream(side):
        for _ in range(4):
            torch.full((want.untyped_storage().nbytes(),), 9, dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    assert torch.equal(copy, want)
    assert ver.error() == 0
