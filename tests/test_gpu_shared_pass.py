"""Passes of requests that go on from one prompt (examples/tree_pass.py): blocks forked by the pool,
groups from the tables, attention that reads the prompt once with the model's form of the scores,
verification, commit.  Every node's target row equals a pass that never speculated nor shared."""

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
    """The toy model's rows after every token of one sequence, in fp64, with its form of the scores."""
    x, q, k, v = (t[0].double() for t in model.projections(torch.tensor(tokens, device="cuda")[None]))
    n, H, K, D = len(tokens), model.heads, model.kv_heads, model.head_dim
    cs = model.table[:n].double()[:, None]

    def turn(t):
        a, b = t[..., :D // 2], t[..., D // 2:]
        return torch.cat([a * cs[..., 0] - b * cs[..., 1], b * cs[..., 0] + a * cs[..., 1]], -1)

    q, k = turn(q), turn(k).repeat_interleave(H // K, 1)
    v = v.repeat_interleave(H // K, 1)
    s = torch.einsum("ihd,jhd->hij", q, k) / D ** 0.5
    if model.softcap:
        s = model.softcap * torch.tanh(s / model.softcap)
    far = torch.arange(n, device="cuda")[:, None] - torch.arange(n, device="cuda")
    if model.slopes is not None:
        s = s - model.slopes.double()[:, None, None] * far
    hidden = far < 0 if model.window is None else (far < 0) | (far >= model.window)
    s = s.masked_fill(hidden, float("-inf"))
    o = torch.einsum("hij,jhd->ihd", s.softmax(-1), v).flatten(1)
    return (x + o @ model.proj.double()) @ model.out.double()


FORMS = {"none": {}, "cap": dict(softcap=2.0), "slopes": dict(slopes=True), "window": dict(window=20),
         "all": dict(softcap=1.5, slopes=True, window=33)}


@pytest.mark.parametrize("kv,tol", [("bf16", 0.03), ("e4m3", 0.08)])
@pytest.mark.parametrize("form", list(FORMS))
def test_rows_equal_a_pass_without_speculation_or_sharing(kv, tol, form):
    """tol: of the rows' root mean square, as for a pass without a form: keys, values, weights and
    outputs are rounded to 8 bits (e4m3: keys and values to 4 significant bits, 2^-4 each, averaged
    over the keys a row sees)."""
    ex = example()
    rng = np.random.default_rng(3)
    s = ex.Session(ex.ToyTarget(**FORMS[form]), batch=5, kv=kv)
    prompt = rng.integers(0, s.m.vocab, 49)
    s.prefill_shared(torch.tensor(prompt, device="cuda"))
    assert (s.table[:, :3] == s.table[0, :3]).all()
    committed = [list(prompt) for _ in range(5)]
    T = torch.full((5,), 0.7, device="cuda")
    for i, shape in enumerate(["binary:3", "random:20", "chain:4", "wide:3,2"]):
        parents, tokens, draft = ex.drafted(s, shape, rng)
        before = [list(c) for c in committed]
        out, logits = s.verify(parents, tokens, draft, temperature=T, seed=i)
        assert s.ver.error() == 0
        par, tok = parents.cpu().numpy(), tokens.cpu().numpy()
        for b in range(5):
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
    # requests have gone their own ways past the prompt, which is still held by all
    groups = s.ver.prefix_groups(s.table, s.seq_len, s.BS, least=s.BS)
    assert groups["length"].tolist() == [48] * 5 and groups["members"].tolist() == [5, 0, 0, 0, 0]
    assert len({tuple(c) for c in committed}) > 1


def test_the_example_runs():
    import subprocess
    import sys
    for more in (["--shared"], ["--shared", "--kv", "bf16", "--softcap", "30", "--slopes"], ["--window", "24"]):
        r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "tree_pass.py"), "--passes", "2", *more],
                           capture_output=True, text=True, timeout=300)
        assert r.returncode == 0 and r.stdout.count("status 0") == 2, r.stdout + r.stderr
