"""The example of a whole verify pass (examples/tree_pass.py): every node's target
row equals a pass that never speculated, and the cache it leaves equals one that
processed the committed tokens alone."""

import importlib.util
import os

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("tree_pass", os.path.join(ROOT, "examples", "tree_pass.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def dense_rows(model, tokens):
    """The toy model's rows after every token of one sequence, in fp64."""
    x, q, k, v = (t[0].double() for t in model.projections(torch.tensor(tokens, device="cuda")[None]))
    n, H, K, D = len(tokens), model.heads, model.kv_heads, model.head_dim
    cs = model.table[:n].double()[:, None]

    def turn(t):
        a, b = t[..., :D // 2], t[..., D // 2:]
        return torch.cat([a * cs[..., 0] - b * cs[..., 1], b * cs[..., 0] + a * cs[..., 1]], -1)

    q, k = turn(q), turn(k).repeat_interleave(H // K, 1)
    v = v.repeat_interleave(H // K, 1)
    s = torch.einsum("ihd,jhd->hij", q, k) / D ** 0.5
    s = s.masked_fill(torch.ones(n, n, device="cuda").triu(1).bool(), float("-inf"))
    o = torch.einsum("hij,jhd->ihd", s.softmax(-1), v).flatten(1)
    return (x + o @ model.proj.double()) @ model.out.double()


@pytest.mark.parametrize("kv,tol", [("bf16", 0.03), ("e4m3", 0.08)])
def test_rows_equal_a_pass_without_speculation(kv, tol):
    """tol: of the rows' root mean square.  Keys, values, weights and outputs
    are rounded to 8 bits (e4m3: keys and values to 4 significant bits, 2^-4 each,
    averaged over the keys a row sees); the rows average several such terms."""
    ex = example()
    rng = np.random.default_rng(3)
    s = ex.Session(ex.ToyTarget(), batch=3, kv=kv)
    prompts = rng.integers(0, s.m.vocab, (3, 38))
    s.prefill(torch.tensor(prompts, device="cuda"))
    committed = [list(p) for p in prompts]  # processed tokens, then the pending one
    T = torch.full((3,), 0.7, device="cuda")
    for i, shape in enumerate(["binary:3", "random:20", "chain:4", "wide:3,2"]):
        parents, tokens, draft = ex.drafted(s, shape, rng)
        before = [list(c) for c in committed]
        out, logits = s.verify(parents, tokens, draft, temperature=T, seed=i)
        assert s.ver.error() == 0
        par, tok = parents.cpu().numpy(), tokens.cpu().numpy()
        for b in range(3):
            for node in range(par.shape[1] + 1):
                path, j = [], node
                while j:
                    path.insert(0, int(tok[b, j - 1]))
                    j = int(par[b, j - 1])
                want = dense_rows(s.m, before[b] + path)[-1]
                err = (logits[b, node].double() - want).pow(2).mean().sqrt() / want.pow(2).mean().sqrt()
                assert err < tol, (shape, b, node, err)
            n = int(out["num_emitted"][b])
            committed[b] += out["out_tokens"][b, :n].tolist()
            assert int(s.seq_len[b]) == len(committed[b]) - 1 and int(s.pending[b]) == committed[b][-1]
    # the cache equals one that processed the committed tokens alone
    for b in range(3):
        fresh = ex.Session(s.m, batch=1, kv=kv)
        fresh.prefill(torch.tensor(committed[b], device="cuda")[None])
        n = len(committed[b]) - 1
        got = torch.empty(1, n, 2, s.m.kv_heads, s.m.head_dim, device="cuda")
        want = torch.empty_like(got)
        zero = torch.zeros(1, dtype=torch.int32, device="cuda")
        s.ver.kv_read(got, zero, kv=s.kv, block_table=s.table[b:b + 1].contiguous())
        fresh.ver.kv_read(want, zero, kv=fresh.kv, block_table=fresh.table)
        # the projections of another batch shape may round differently in the library product
        assert (got - want).abs().max() <= 2.0 ** -3 * want.abs().max()
        assert ((got - want).abs() > 1e-6).float().mean() < 0.02


def test_grammar_masks_bind_the_emitted_tokens():
    ex = example()
    rng = np.random.default_rng(5)
    s = ex.Session(ex.ToyTarget(), batch=4, kv="bf16")
    s.prefill(torch.tensor(rng.integers(0, s.m.vocab, (4, 9)), device="cuda"))
    parents, tokens, draft = ex.drafted(s, "binary:2", rng)
    allowed = torch.zeros(4, parents.shape[1] + 1, s.m.vocab // 32, dtype=torch.int32, device="cuda")
    allowed[:, :, 3] = 0x00FF0000  # tokens 112 .. 119
    out, logits = s.verify(parents, tokens, draft, temperature=torch.ones(4, device="cuda"), allowed=allowed, seed=9)
    assert s.ver.error() == 0
    emitted = out["out_tokens"].gather(1, (out["num_emitted"].long() - 1)[:, None]).flatten()
    assert ((emitted >= 112) & (emitted < 120)).all()
    assert torch.isinf(logits).sum(-1).eq(s.m.vocab - 8).all()
