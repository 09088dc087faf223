"""One verify pass of a token tree, from drafted tokens to the committed cache.

A toy model of one attention layer with random weights stands in for the target:
what matters is the order of the calls and what each hands to the next.

    tree_mask        the trees' ancestor bits and depths, once a pass
    kv_append        queries and keys rotated to the nodes' positions, the nodes'
                     entries written to the staging buffer in the cache's format
    tree_attention   the nodes over the committed cache and their own ancestors
    adjust_logits    penalties and grammar masks on every node's row
    verify_tree      the accepted path and the next token
    kv_commit_tree   the path's entries moved into the paged cache
    commit_rollback  lengths, blocks and reference counts

    python examples/tree_pass.py [--kv bf16|e4m3] [--passes N]
"""

import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from speculative_decoding_verification_07_gb300 import binding, rope, workloads  # noqa: E402


class ToyTarget:
    """tied embedding -> one attention layer (grouped heads, rotary) -> logits."""

    def __init__(self, vocab=512, width=256, heads=4, kv_heads=2, head_dim=64, seed=0, device="cuda"):
        g = torch.Generator(device).manual_seed(seed)
        self.heads, self.kv_heads, self.head_dim, self.vocab = heads, kv_heads, head_dim, vocab

        def weight(*shape):
            return (torch.randn(*shape, generator=g, device=device) / shape[0] ** 0.5).bfloat16()

        self.embedding = weight(vocab, width) * vocab ** 0.5
        self.qkv = weight(width, (heads + 2 * kv_heads) * head_dim)
        self.proj = weight(heads * head_dim, width)
        self.out = weight(width, vocab)
        self.table = rope.rope_table(4096, rope.rope_frequencies(head_dim), device=device)

    def projections(self, tokens):
        """Queries, keys and values [B, R, heads, head_dim]: slices of one product."""
        x = self.embedding[tokens.long()]
        y = (x @ self.qkv).unflatten(-1, (-1, self.head_dim))
        H, K = self.heads, self.kv_heads
        return x, y[:, :, :H], y[:, :, H:H + K], y[:, :, H + K:]

    def logits(self, x, attended):
        return (x + attended.flatten(2) @ self.proj) @ self.out


class Session:
    """The serving state of a batch: paged cache, tables, lengths, histories."""

    def __init__(self, model, batch=4, kv="bf16", block_size=16, blocks=256, max_blocks=32, device="cuda"):
        self.m, self.B, self.BS, self.nb, self.device = model, batch, block_size, blocks, device
        self.ver = binding.Verifier(0)
        row = model.head_dim + (binding.E4M3_TAIL if kv == "e4m3" else 0)
        self.dtype = torch.uint8 if kv == "e4m3" else torch.bfloat16
        self.kv = torch.zeros(blocks, 1, 2, model.kv_heads, block_size, row, dtype=self.dtype, device=device)
        self.pool = binding.BlockPool(self.ver.handle, blocks, block_size)
        self.table = torch.full((batch, max_blocks), -1, dtype=torch.int32, device=device)
        self.seq_len = torch.zeros(batch, dtype=torch.int32, device=device)
        self.history = torch.full((batch, 512), -1, dtype=torch.int32, device=device)  # tokens emitted so far
        self.emitted = 0

    def prefill(self, prompts):
        """prompts [B, P]: all but the last token are processed into the cache; the last is pending."""
        self.pending = prompts[:, -1:].int().contiguous()
        done = prompts[:, :-1].int().contiguous()
        R = done.shape[1]
        more = torch.full((self.B,), R - 1, dtype=torch.int32, device=self.device)
        self.pool.reserve(self.seq_len, more, self.table)
        _, _, k, v = self.m.projections(done)
        self.ver.kv_append(k, v, self.seq_len, kv=self.kv, block_table=self.table, rope=self.m.table)
        self.seq_len += R

    def verify(self, parents, tokens, draft, *, temperature, rep_penalty=None, allowed=None, seed=0):
        """parents [B, N], tokens [B, N]: the drafted trees; draft [B, N + 1, V]: the draft's rows.
        Returns the verified step's outputs and the adjusted target rows."""
        m, ver, B, N = self.m, self.ver, self.B, parents.shape[1]
        tree = ver.tree_mask(parents)
        depth = int(tree["depth"].max())  # the longest path any tree can give
        lookahead = torch.full((B,), depth, dtype=torch.int32, device=self.device)
        self.pool.reserve(self.seq_len, lookahead, self.table)

        x, q, k, v = m.projections(torch.cat([self.pending, tokens], 1))
        stage = torch.empty(B, N + 1, 1, 2, m.kv_heads, self.kv.shape[-1], dtype=self.dtype, device=self.device)
        q = ver.kv_append(k, v, self.seq_len, q=q, stage=stage, rope=m.table, depth=tree["depth"])
        attended = ver.tree_attention(q, self.kv, self.table, self.seq_len, stage=stage, mask=tree["mask"])
        logits = m.logits(x, attended).contiguous()
        ver.adjust_logits(logits, history=self.history, tokens=tokens, mask=tree["mask"], rep_penalty=rep_penalty,
                          allowed=allowed)

        out = ver.verify_tree(target=logits, draft=draft, parent=parents, tokens=tokens, temperature=temperature,
                              seed=seed, seq_len=self.seq_len)
        binding.kv_commit_tree(ver.handle, out["accepted"], out["path"], self.seq_len, self.table, self.BS, self.nb, stage,
                               self.kv, depth)
        self.pool.commit_rollback(lookahead, out["accepted"], self.seq_len, self.table)
        # histories and the new pending tokens
        n = out["num_emitted"].long()
        self.pending = out["out_tokens"].gather(1, (n - 1)[:, None]).contiguous()
        width = min(N + 1, self.history.shape[1] - self.emitted)
        self.history[:, self.emitted:self.emitted + width] = out["out_tokens"][:, :width]  # -1 past the last
        self.emitted += width
        return out, logits


def drafted(session, shape, rng):
    """Trees of a named shape with random proposals, and the (uniform) draft's rows."""
    par = workloads.tree_shape(shape, rng)
    B, N, V = session.B, len(par), session.m.vocab
    parents = torch.tensor(np.tile(np.array(par, np.int32), (B, 1)), device=session.device)
    tokens = torch.tensor(rng.integers(0, V, (B, N)).astype(np.int32), device=session.device)
    return parents, tokens, torch.zeros(B, N + 1, V, dtype=torch.bfloat16, device=session.device)


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--kv", choices=("bf16", "e4m3"), default="e4m3")
    ap.add_argument("--passes", type=int, default=4)
    a = ap.parse_args()
    rng = np.random.default_rng(0)
    s = Session(ToyTarget(), kv=a.kv)
    s.prefill(torch.tensor(rng.integers(0, s.m.vocab, (s.B, 41)), device="cuda"))
    T = torch.full((s.B,), 0.8, device="cuda")
    for i in range(a.passes):
        out, _ = s.verify(*drafted(s, "binary:3", rng), temperature=T, rep_penalty=torch.full((s.B,), 1.2, device="cuda"),
                          seed=i)
        print(f"pass {i}: accepted {out['accepted'].tolist()}, pending {s.pending.flatten().tolist()}, "
              f"lengths {s.seq_len.tolist()}, status {s.ver.error()}")


if __name__ == "__main__":
    main()
