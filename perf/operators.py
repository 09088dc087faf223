"""The operators around the verification step, as cases to time and compare.

Four operators serve one verify pass of speculative decoding:

  mask       a token tree's parents -> every node's ancestor bits and depth
  cache      rotary positions, K/V entries written into the paged cache or the staging buffer
             (bf16, fp32, or e4m3 with a power-of-two scale per entry and head), and read back
  attention  the tree's queries over the paged cache and the tree's own staged entries
  logits     penalties, biases and grammar masks on the target's rows

`own = False` runs them in elementary torch operations in 32 bits; `own = True` through the
package's public calls.  Sizes are those of the repository's own workloads: 4 heads x d64 fp32,
8 KV heads x d128 and 4 KV heads x d128 bf16 with paged blocks of 16, vocabularies 1024, 32000,
128256 and 151936, batches 1 to 256, prefixes up to 8192, trees of the named shapes.
"""

import math
import random

import numpy as np
import torch

own = False

E4M3_TAIL = 16  # bytes after an entry's codes: its fp32 scale, then zeros


# --------------------------------------------------------------------------- #
# shapes
# --------------------------------------------------------------------------- #
def tree_parents(shape):
    """parent[i - 1] of node i (0: the pending token); random trees depend on the shape alone."""
    kind, arg = shape.split(":")
    if kind == "chain":
        return list(range(int(arg)))
    if kind == "binary":
        par, level = [], [0]
        for _ in range(int(arg)):
            nxt = []
            for p in level:
                for _ in range(2):
                    par.append(p)
                    nxt.append(len(par))
            level = nxt
        return par
    if kind == "wide":
        w, d = (int(x) for x in arg.split(","))
        par = []
        for _ in range(w):
            par.append(0)
            for _ in range(d - 1):
                par.append(len(par))
        return par
    r = random.Random(int(arg))
    return [r.randrange(i) for i in range(1, int(arg) + 1)]


def lengths(case):
    """The requests' prefix lengths: spread evenly over [lo, hi], in an order of their own."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    s = [lo + (hi - lo) * b // max(1, B - 1) for b in range(B)] if B > 1 else [hi]
    random.Random(B * 7919 + hi).shuffle(s)
    return s


def nodes_of(case):
    """n_b per request: the whole tree, or (ragged) any count down to none."""
    N = len(tree_parents(case["tree"]))
    if not case.get("ragged"):
        return [N] * case["B"]
    r = random.Random(case["B"] * 31 + N)
    return [r.randrange(N + 1) for _ in range(case["B"])]


def entry_bytes(case):
    D = case["D"]
    return {"bf16": 2 * D, "fp32": 4 * D, "e4m3": D + E4M3_TAIL}[case["kv"]]


# --------------------------------------------------------------------------- #
# cases
# --------------------------------------------------------------------------- #
def listed():
    return [
        # one request's smallest verify step: fp32 heads of 64, five drafts in a chain, 32 cached tokens
        dict(name="attend_fp32_b1", op="attention", B=1, lo=32, hi=32, Hq=4, Hkv=4, D=64, kv="fp32",
             tree="chain:5", staged=True, ragged=False, bs=16),
        # one user's next token: a single query row over a few hundred cached positions
        dict(name="attend_token_b1", op="attention", B=1, lo=777, hi=777, Hq=32, Hkv=8, D=128, kv="bf16",
             tree="chain:0", staged=False, ragged=False, bs=16),
        # a serving batch without drafts: single tokens over ragged prefixes
        dict(name="attend_token_b64", op="attention", B=64, lo=128, hi=8192, Hq=32, Hkv=8, D=128, kv="bf16",
             tree="chain:0", staged=False, ragged=False, bs=16),
        # the same batch with a binary tree of depth 3 per request
        dict(name="attend_tree_b64", op="attention", B=64, lo=128, hi=8192, Hq=32, Hkv=8, D=128, kv="bf16",
             tree="binary:3", staged=True, ragged=False, bs=16),
        # the same over a quantised cache
        dict(name="attend_tree_e4m3", op="attention", B=64, lo=128, hi=8192, Hq=32, Hkv=8, D=128, kv="e4m3",
             tree="binary:3", staged=True, ragged=False, bs=16),
        # few requests with long prefixes and large ragged trees, an odd head group (28 over 4)
        dict(name="attend_long_wide", op="attention", B=4, lo=20001, hi=65536, Hq=28, Hkv=4, D=128, kv="bf16",
             tree="random:63", staged=True, ragged=True, bs=16),
        # the trees of a serving batch, staged in 8 bits until the walk has chosen a path
        dict(name="cache_tree_e4m3", op="cache", B=64, lo=128, hi=8192, Hq=32, Hkv=8, D=128, kv="e4m3",
             tree="binary:3", staged=True, ragged=True, bs=16, rot=128, pairs=False),
        # prompts of four requests, rotated in pairs over half of the head, into the 8-bit pages
        dict(name="cache_prompt_e4m3", op="cache", B=4, lo=0, hi=4097, Hq=32, Hkv=8, D=128, kv="e4m3",
             tree="chain:2040", staged=False, ragged=False, bs=16, rot=64, pairs=True),
        # the rows of one small request, every rule on
        dict(name="logits_fp32_b1", op="logits", B=1, V=1024, kind="fp32", tree="chain:5", ragged=False,
             history=37, bias=5, grammar=True),
        # the rows of a serving batch of trees
        dict(name="logits_tree_b64", op="logits", B=64, V=128256, kind="bf16", tree="binary:2", ragged=False,
             history=1500, bias=64, grammar=True),
        # the tree of one request, once a step
        dict(name="mask_b1", op="mask", B=1, tree="random:14", ragged=False),
        # large ragged trees of a large batch, once a step
        dict(name="mask_b256", op="mask", B=256, tree="random:127", ragged=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _tree(rng, most):
    kind = rng.choice(["chain", "binary", "wide", "random"])
    if kind == "binary":
        return "binary:%d" % rng.randint(1, max(1, int(math.log2(most + 2)) - 1))
    if kind == "wide":
        w = rng.randint(1, max(1, min(8, most)))
        return "wide:%d,%d" % (w, rng.randint(1, max(1, most // w)))
    return "%s:%d" % (kind, rng.randint(0, most) if kind == "chain" else _log(rng, 1, most))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "cache", "cache", "logits", "logits", "mask"])
    if op == "mask":
        return dict(op=op, B=_log(rng, 1, 256), tree="random:%d" % _log(rng, 9, 127),
                    ragged=rng.random() < 0.5)
    if op == "logits":
        V = rng.choice([1024, 4093, 32000, 128256, 151936])
        tree = _tree(rng, 14)
        B = _log(rng, 1, max(1, min(256, 64 * 7 * 128256 // (V * (len(tree_parents(tree)) + 1)))))
        return dict(op=op, B=B, V=V, kind=rng.choice(["bf16", "bf16", "fp32"]) if V * B < 1e6 else "bf16",
                    tree=tree, ragged=rng.random() < 0.5, history=rng.randint(0, 1500),
                    bias=rng.choice([0, rng.randint(1, 64)]), grammar=rng.random() < 0.7)
    Hq, Hkv, D = rng.choice([(32, 8, 128), (28, 4, 128), (8, 8, 64), (16, 2, 64), (32, 8, 128)])
    kv = rng.choice(["bf16", "e4m3", "bf16", "e4m3", "fp32"])
    bs = rng.choice([16, 16, 16, 32, 64, 8])
    if op == "cache":
        tree = "chain:%d" % _log(rng, 1, 2040) if rng.random() < 0.4 else _tree(rng, 63)
        most = 4 * 2041 // (len(tree_parents(tree)) + 1) // (2 if kv == "fp32" else 1)
        B = _log(rng, 1, max(1, min(64, most)))
        hi = _log(rng, 1, 8192)
        return dict(op=op, B=B, lo=rng.randint(0, hi), hi=hi, Hq=Hq, Hkv=Hkv, D=D, kv=kv, tree=tree,
                    staged=rng.random() < 0.5, ragged=rng.random() < 0.5, bs=bs,
                    rot=rng.choice([D, D, D // 2, 0]), pairs=rng.random() < 0.4)
    if kv == "fp32":  # the fp32 cache is the small configuration's
        B, hi, Hq, Hkv, D = _log(rng, 1, 8), _log(rng, 1, 512), 4, 4, 64
        return dict(op=op, B=B, lo=rng.randint(0, hi), hi=hi, Hq=Hq, Hkv=Hkv, D=D, kv=kv, tree=_tree(rng, 14),
                    staged=rng.random() < 0.5, ragged=rng.random() < 0.5, bs=bs)
    B = _log(rng, 1, 64)
    hi = _log(rng, 1, min(65536, 64 * 4096 // B))
    tree = "chain:0" if rng.random() < 0.3 else _tree(rng, 63 if B * hi <= 1 << 17 else 14)
    return dict(op=op, B=B, lo=rng.randint(0, hi), hi=hi, Hq=Hq, Hkv=Hkv, D=D, kv=kv, tree=tree,
                staged=rng.random() < 0.6, ragged=rng.random() < 0.4, bs=bs)


# --------------------------------------------------------------------------- #
# inputs
# --------------------------------------------------------------------------- #
LAYERS, LAYER = 2, 1  # the cache holds two layers; a pass works on the second


def _entries(shape, kv, D, gen):
    """Random K/V entries [..., D] of a format; the keys' channels are not all alike in size."""
    dev = gen.device
    if kv == "e4m3":
        out = torch.zeros(*shape, D + E4M3_TAIL, dtype=torch.uint8, device=dev)
        x = torch.randn(*shape, D, generator=gen, device=dev, dtype=torch.bfloat16)
        out[..., :D] = x.mul_(70).to(torch.float8_e4m3fn).view(torch.uint8)
        e = torch.randint(-8, -5, tuple(shape), generator=gen, device=dev)
        out[..., D:D + 4] = torch.exp2(e.float()).unsqueeze(-1).view(torch.uint8)
        return out
    gain = torch.exp2(0.5 * torch.randn(D, generator=gen, device=dev))
    x = torch.randn(*shape, D, generator=gen, device=dev, dtype=torch.bfloat16 if kv == "bf16" else torch.float32)
    x *= gain.to(x.dtype)
    return x


def _table(case, gen, blocks_for):
    """Block tables over a pool whose blocks are handed out in random order; -1 past the last."""
    n = [-(-x // case["bs"]) for x in blocks_for]
    total, width = max(1, sum(n)), max(1, max(n))
    order = torch.randperm(total, generator=gen, device=gen.device).int()
    table = torch.full((case["B"], width), -1, dtype=torch.int32, device=gen.device)
    at = 0
    for b, m in enumerate(n):
        table[b, :m] = order[at:at + m]
        at += m
    return table, total


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _pack(bits):
    """[..., n] truth values -> [..., ceil(n / 32)] int32 words, bit j of word w standing for 32 w + j."""
    n = bits.shape[-1]
    bits = torch.nn.functional.pad(bits, (0, -n % 32)).reshape(*bits.shape[:-1], -1, 32)
    words = (bits.long() << torch.arange(32, device=bits.device)).sum(-1)
    return torch.where(words >= 1 << 31, words - (1 << 32), words).int()


def _unpack(words, n):
    return ((words.unsqueeze(-1) >> torch.arange(32, device=words.device, dtype=torch.int32)) & 1).flatten(-2)[..., :n].bool()


def _ancestors(par):
    """(bits, depth) of one tree, on the host."""
    n = len(par) + 1
    a = np.zeros((n, n), bool)
    depth = np.zeros(n, np.int32)
    a[0, 0] = True
    for i in range(1, n):
        a[i] = a[par[i - 1]]
        a[i, i] = True
        depth[i] = depth[par[i - 1]] + 1
    return a, depth


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    par = tree_parents(case["tree"])
    B, N, R = case["B"], len(par), len(par) + 1
    s = dict(case=case, B=B, N=N, R=R, n_nodes=_ints(nodes_of(case)))
    if case["op"] == "mask":
        # every request its own tree: each node under an earlier one, drawn by the seed
        p = torch.rand(B, N, generator=gen, device="cuda") * torch.arange(1, R, device="cuda")
        s["parent"] = p.int().contiguous()
        return s
    bits, depth = _ancestors(par)
    n = torch.tensor(nodes_of(case), device="cuda")
    alive = torch.arange(R, device="cuda") <= n[:, None]
    s["mask"] = _pack(torch.tensor(bits, device="cuda") & alive[:, :, None]).contiguous()
    s["depth"] = (torch.tensor(depth, device="cuda") * alive).int().contiguous()
    if case["op"] == "logits":
        V, dt = case["V"], torch.bfloat16 if case["kind"] == "bf16" else torch.float32
        ld = -(-V // 8) * 8
        s["logits"] = (torch.randn(B, R, ld, generator=gen, device="cuda") * 3).to(dt)
        s["out"] = torch.empty_like(s["logits"])
        zipf = torch.rand(B, case["history"] + N + case["bias"], generator=gen, device="cuda")
        ids = (V ** zipf - 1).long().clamp(0, V - 1).int()  # small ids are the frequent ones
        s["history"] = ids[:, :case["history"]].contiguous()
        s["tokens"] = ids[:, case["history"]:case["history"] + N].contiguous()
        step = torch.rand(B, max(1, case["bias"]), generator=gen, device="cuda") * (V // max(1, case["bias"]) - 1)
        s["bias_ids"] = (step.long() + torch.arange(case["bias"] or 1, device="cuda") * (V // max(1, case["bias"]))).int()
        s["bias_values"] = torch.randn(B, max(1, case["bias"]), generator=gen, device="cuda") * 4
        r = torch.rand(3, B, generator=gen, device="cuda")
        s["rep"], s["presence"], s["frequency"] = 1 + r[0] * 0.5, r[1] - 0.25, r[2] * 0.5
        if case["grammar"]:  # rows allow a few, most or nearly all tokens
            keep = torch.rand(B, R, 1, generator=gen, device="cuda") ** 2
            W = -(-V // 32)
            s["allowed"] = torch.empty(B, R, W, dtype=torch.int32, device="cuda")
            for b in range(0, B, 8):
                s["allowed"][b:b + 8] = _pack(torch.rand(keep[b:b + 8].shape[0], R, V, generator=gen, device="cuda") >= keep[b:b + 8])
        return s
    Hq, Hkv, D, kv = case["Hq"], case["Hkv"], case["D"], case["kv"]
    dt = torch.float32 if kv == "fp32" else torch.bfloat16
    S = lengths(case)
    s["seq_len"] = _ints(S)
    more = 0 if case["staged"] else R
    s["table"], blocks = _table(case, gen, [x + more for x in S])
    E = (blocks, LAYERS, 2, Hkv, case["bs"])
    if case["op"] == "cache":
        s["kv"] = torch.zeros(*E, D + E4M3_TAIL, dtype=torch.uint8, device="cuda") if kv == "e4m3" else \
            torch.zeros(*E, D, dtype=dt, device="cuda")
        if case["staged"]:
            s["kv"] = torch.zeros(B, R, LAYERS, 2, Hkv, s["kv"].shape[-1], dtype=s["kv"].dtype, device="cuda")
        # one projection's output holds a token's queries, keys and values side by side
        s["qkv"] = torch.randn(B, R, Hq + 2 * Hkv, D, generator=gen, device="cuda", dtype=dt)
        s["q_out"] = torch.empty(B, R, Hq, D, dtype=dt, device="cuda")
        s["read"] = torch.empty(B, R, 2, Hkv, D, dtype=dt, device="cuda")
        s["rope"] = None
        if case["rot"]:
            inv = 10000.0 ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64, device="cuda") / case["rot"])
            ang = torch.arange(case["hi"] + R + 1, dtype=torch.float64, device="cuda")[:, None] * inv
            s["rope"] = torch.stack([ang.cos(), ang.sin()], -1).float().contiguous()
        return s
    s["kv"] = _entries(E, kv, D, gen)
    s["stage"] = _entries((B, R, LAYERS, 2, Hkv), kv, D, gen) if case["staged"] else None
    s["q"] = torch.randn(B, R, Hq, D, generator=gen, device="cuda", dtype=dt)
    s["out"] = torch.empty_like(s["q"])
    return s


# --------------------------------------------------------------------------- #
# plain forms: elementary operations in 32 bits
# --------------------------------------------------------------------------- #
def _decode(x, kv, D):
    if kv != "e4m3":
        return x.float()
    scale = x[..., D:D + 4].contiguous().view(torch.float32)
    return x[..., :D].view(torch.float8_e4m3fn).float() * scale


def _plain_mask(s):
    B, R = s["B"], s["R"]
    i = torch.arange(R, device="cuda")
    up = torch.eye(R, device="cuda").repeat(B, 1, 1)
    if s["N"]:
        up[:, 1:].scatter_(2, s["parent"].long().unsqueeze(-1), 1.0)
    k = 1
    while k < R:  # ancestors within 2 k steps
        up = (up @ up > 0).float()
        k *= 2
    bits = (up > 0) & (i <= s["n_nodes"][:, None])[:, :, None]
    return {"mask": _pack(bits), "depth": (bits.sum(-1) - 1).clamp(min=0).int()}


def _rotate(x, cs, pairs):
    """x [B, R, H, D]; cs [B, R, rot / 2, 2]."""
    if cs is None:
        return x
    c, s = cs[..., 0].unsqueeze(2), cs[..., 1].unsqueeze(2)
    rot = 2 * c.shape[-1]
    r = x[..., :rot]
    a, b = (r[..., 0::2], r[..., 1::2]) if pairs else (r[..., :rot // 2], r[..., rot // 2:])
    a, b = a * c - b * s, b * c + a * s
    r = torch.stack([a, b], -1).flatten(-2) if pairs else torch.cat([a, b], -1)
    return torch.cat([r, x[..., rot:]], -1)


def _encode(x, kv):
    """fp32 [..., D] -> entries of a format."""
    if kv == "fp32":
        return x
    if kv == "bf16":
        return x.to(torch.bfloat16)
    amax = x.abs().amax(-1, keepdim=True)
    m, e = torch.frexp(amax)  # amax = m 2^e with m in [1/2, 1); 448 = 0.875 * 2^9
    e = torch.where(m <= 0.875, e - 9, e - 8)
    scale = torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e), torch.ones_like(amax))
    codes = (x / scale).to(torch.float8_e4m3fn).view(torch.uint8)
    tail = torch.zeros(*x.shape[:-1], E4M3_TAIL, dtype=torch.uint8, device=x.device)
    tail[..., :4] = scale.contiguous().view(torch.uint8)
    return torch.cat([codes, tail], -1)


def _plain_cache(s):
    c, R, D = s["case"], s["R"], s["case"]["D"]
    x = s["qkv"].float()
    q, k, v = x[:, :, :c["Hq"]], x[:, :, c["Hq"]:c["Hq"] + c["Hkv"]], x[:, :, c["Hq"] + c["Hkv"]:]
    cs = None if s["rope"] is None else s["rope"][(s["seq_len"][:, None] + s["depth"]).long()]
    live = (torch.arange(R, device="cuda") <= s["n_nodes"][:, None])
    q_out = _rotate(q, cs, c["pairs"]) * live[:, :, None, None]
    e = _encode(torch.stack([_rotate(k, cs, c["pairs"]), v], 2), c["kv"])  # [B, R, 2, H, E]
    b, i = live.nonzero(as_tuple=True)
    if c["staged"]:
        s["kv"][b, i, LAYER] = e[b, i]
        back = s["kv"][:, :, LAYER]
    else:
        p = s["seq_len"].long()[:, None] + torch.arange(R, device="cuda")
        blk, slot = s["table"].long().gather(1, p // c["bs"]), p % c["bs"]
        s["kv"][blk[b, i], LAYER, :, :, slot[b, i]] = e[b, i]
        back = s["kv"][blk, LAYER, :, :, slot]
    back = _decode(back, c["kv"], D) * live[:, :, None, None, None]
    return {"q": q_out.to(s["qkv"].dtype), "kv": back.to(s["read"].dtype)}


def _plain_attention(s):
    c, B, R, D, bs = s["case"], s["B"], s["R"], s["case"]["D"], s["case"]["bs"]
    H, G = c["Hkv"], c["Hq"] // c["Hkv"]
    pages = _decode(s["kv"][s["table"].long().clamp(min=0), LAYER], c["kv"], D)  # [B, m, 2, H, bs, D]
    kv = pages.permute(2, 0, 3, 1, 4, 5).reshape(2, B, H, -1, D)
    at = torch.arange(kv.shape[3], device="cuda") - s["seq_len"][:, None]  # 0 is the pending token
    bits = _unpack(s["mask"], R) & (torch.arange(R, device="cuda") <= s["n_nodes"][:, None])[:, None]
    if c["staged"]:
        kv = torch.cat([kv, _decode(s["stage"][:, :, LAYER], c["kv"], D).permute(2, 0, 3, 1, 4)], 3)
        seen = torch.cat([(at < 0)[:, None].expand(B, R, -1), bits], 2)
    else:
        seen = (at < 0)[:, None] | ((at < R)[:, None] & bits.gather(2, at.clamp(0, R - 1)[:, None].expand(B, R, -1)))
    q = s["q"].float().reshape(B, R, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, R * G, D)
    x = (q @ kv[0].transpose(2, 3) / math.sqrt(D)).reshape(B, H, R, G, -1)
    x = x.masked_fill_(~seen[:, None, :, None], -math.inf)
    x -= x.amax(-1, keepdim=True).clamp(min=-3e38)
    x = x.exp_().reshape(B, H, R * G, -1)
    o = (x @ kv[1]) / x.sum(-1, keepdim=True).clamp(min=1e-30)
    o = o.reshape(B, H, R, G, D).permute(0, 2, 1, 3, 4).reshape(B, R, c["Hq"], D)
    return (o * (torch.arange(R, device="cuda") <= s["n_nodes"][:, None])[:, :, None, None]).to(s["q"].dtype)


def _plain_logits(s):
    c, B, R, N, V = s["case"], s["B"], s["R"], s["N"], s["case"]["V"]
    count = torch.zeros(B, 1, V, device="cuda")
    count.scatter_add_(2, s["history"].long()[:, None], torch.ones(B, 1, c["history"], device="cuda"))
    count = count.repeat(1, R, 1)
    if N:
        path = _unpack(s["mask"], R)[:, :, 1:].float()
        count.scatter_add_(2, s["tokens"].long()[:, None].expand(B, R, N), path)
    rep, pres, freq = (s[k][:, None, None] for k in ("rep", "presence", "frequency"))
    x = s["logits"][:, :, :V].float()
    x = torch.where(count > 0, torch.where(x > 0, x / rep, x * rep) - (freq * count + pres), x)
    if c["bias"]:
        x.scatter_add_(2, s["bias_ids"].long()[:, None].expand(B, R, -1), s["bias_values"][:, None].expand(B, R, -1))
    if c["grammar"]:
        x.masked_fill_(~_unpack(s["allowed"], V), -math.inf)
    live = (torch.arange(R, device="cuda") <= s["n_nodes"][:, None])[:, :, None]
    return torch.where(live, x, s["logits"][:, :, :V].float()).to(s["logits"].dtype)


# --------------------------------------------------------------------------- #
# the package's calls
# --------------------------------------------------------------------------- #
_verifier = None


def _handle():
    global _verifier
    if _verifier is None:
        from speculative_decoding_verification_07_gb300 import binding
        _verifier = binding.Verifier(0)
    return _verifier


def _own(s):
    ver, c = _handle(), s["case"]
    if c["op"] == "mask":
        return ver.tree_mask(s["parent"], n_nodes=s["n_nodes"])
    if c["op"] == "attention":
        return ver.tree_attention(s["q"], s["kv"], s["table"], s["seq_len"], layer=LAYER, stage=s["stage"],
                                  mask=s["mask"], n_nodes=s["n_nodes"], out=s["out"])
    if c["op"] == "logits":
        more = dict(bias_ids=s["bias_ids"], bias_values=s["bias_values"]) if c["bias"] else {}
        out = ver.adjust_logits(s["logits"], V=c["V"], out=s["out"], history=s["history"], tokens=s["tokens"],
                                mask=s["mask"], n_nodes=s["n_nodes"], rep_penalty=s["rep"], presence=s["presence"],
                                frequency=s["frequency"], allowed=s.get("allowed"), **more)
        return out[:, :, :c["V"]]
    Hq, Hkv = c["Hq"], c["Hkv"]
    q, k, v = s["qkv"][:, :, :Hq], s["qkv"][:, :, Hq:Hq + Hkv], s["qkv"][:, :, Hq + Hkv:]
    place = dict(stage=s["kv"]) if c["staged"] else dict(kv=s["kv"], block_table=s["table"])
    ver.kv_append(k, v, s["seq_len"], layer=LAYER, q=q, q_out=s["q_out"], rope=s["rope"], interleaved=c["pairs"],
                  depth=s["depth"], n_nodes=s["n_nodes"], **place)
    ver.kv_read(s["read"], s["seq_len"], layer=LAYER, n_nodes=s["n_nodes"], **place)
    return {"q": s["q_out"], "kv": s["read"]}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    return {"mask": _plain_mask, "cache": _plain_cache, "attention": _plain_attention, "logits": _plain_logits}[op](state)


# --------------------------------------------------------------------------- #
# what a pass cannot do without
# --------------------------------------------------------------------------- #
def work(case):
    par = tree_parents(case["tree"])
    B, R, nodes = case["B"], len(par) + 1, nodes_of(case)
    if case["op"] == "mask":
        W = -(-R // 32)
        return {"bytes": 4 * B * (len(par) + 1 + R * (W + 1)), "flops": 0}
    rows = sum(n + 1 for n in nodes)
    if case["op"] == "logits":
        V, eb = case["V"], 2 if case["kind"] == "bf16" else 4
        ids = case["history"] + len(par) + 2 * case["bias"]
        return {"bytes": 2 * B * R * V * eb + (rows * V // 8 if case["grammar"] else 0) + 4 * B * ids, "flops": 4 * rows * V}
    eb = 4 if case["kv"] == "fp32" else 2
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    if case["op"] == "cache":
        new = rows * 2 * Hkv
        table = min(case["hi"] + R, rows) * case["rot"] * 4
        moved = rows * 2 * Hq * D * eb + new * (D * eb + entry_bytes(case)) + table
        back = new * (entry_bytes(case) + D * eb)
        return {"bytes": moved + back, "flops": 3 * rows * (Hq + Hkv) * case["rot"]}
    a, _ = _ancestors(par)
    S = lengths(case)
    keys = sum(s + n + 1 for s, n in zip(S, nodes))
    pairs = sum((n + 1) * s + int(a[:n + 1].sum()) for s, n in zip(S, nodes))
    return {"bytes": keys * 2 * Hkv * entry_bytes(case) + 2 * rows * Hq * D * eb, "flops": 4 * D * Hq * pairs}


# --------------------------------------------------------------------------- #
# the definitions in 64 bits
# --------------------------------------------------------------------------- #
def _e4m3_values():
    """The 256 values of the 8-bit format: sign, 4 exponent bits with bias 7, 3 fraction bits."""
    v = np.empty(256)
    for code in range(256):
        e, f = (code >> 3) & 15, code & 7
        x = f * 2.0 ** -9 if e == 0 else (8 + f) * 2.0 ** (e - 10)
        x = math.nan if (code & 127) == 127 else x
        v[code] = -x if code & 128 else x
    return torch.tensor(v, device="cuda")


def _values(entries, kv, D):
    if kv != "e4m3":
        return entries.double()
    b = entries[..., D:D + 4].long()
    bits = b[..., 0] | b[..., 1] << 8 | b[..., 2] << 16 | b[..., 3] << 24
    scale = torch.exp2(((bits >> 23) & 255).double() - 127) * (1 + (bits & 0x7FFFFF).double() / (1 << 23))
    return _e4m3_values()[entries[..., :D].long()] * scale.unsqueeze(-1)


def _to_e4m3(y):
    """The nearest of the format's values (even fractions on ties), in 64 bits."""
    e = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    return (torch.round(y / step) * step).clamp(-448, 448)


def exact(case, seed):
    s = prepare(case, seed)
    B, R, nodes = s["B"], s["R"], nodes_of(case)
    if case["op"] == "mask":
        return None  # whole numbers: the plain form's have to be met
    anc, depth = _ancestors(tree_parents(case["tree"]))
    anc = torch.tensor(anc, device="cuda")
    if case["op"] == "logits":
        V = case["V"]
        out = torch.empty(B, R, V, dtype=torch.float64, device="cuda")
        for b in range(B):
            for j in range(R):
                x = s["logits"][b, j, :V].double()
                if j <= nodes[b]:
                    ids = torch.cat([s["history"][b], s["tokens"][b][anc[j, 1:]]]).long()
                    n = torch.bincount(ids, minlength=V).double()
                    rep = s["rep"][b].double()
                    y = torch.where(x > 0, x / rep, x * rep) - s["frequency"][b].double() * n - s["presence"][b].double()
                    x = torch.where(n > 0, y, x)
                    if case["bias"]:
                        x.index_add_(0, s["bias_ids"][b].long(), s["bias_values"][b].double())
                    if case["grammar"]:
                        t = torch.arange(V, device="cuda")
                        x[(s["allowed"][b, j].long()[t // 32] >> (t % 32)) & 1 == 0] = -math.inf
                out[b, j] = x
        return out
    Hq, Hkv, D, S = case["Hq"], case["Hkv"], case["D"], lengths(case)
    G = Hq // Hkv
    if case["op"] == "cache":
        x = s["qkv"].double()
        pos = torch.tensor(S, device="cuda")[:, None] + torch.tensor(depth, device="cuda")
        for b in range(B):
            x[b, nodes[b] + 1:] = 0
        half = case["rot"] // 2
        if half:
            inv = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
            z = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), pos.double()[..., None] * inv)[:, :, None]
            r = x[:, :, :Hq + Hkv, :2 * half]
            first, second = (slice(0, None, 2), slice(1, None, 2)) if case["pairs"] else (slice(0, half), slice(half, None))
            w = torch.complex(r[..., first], r[..., second]) * z
            r[..., first], r[..., second] = w.real, w.imag
        kv = torch.stack([x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:]], 2)
        if case["kv"] == "e4m3":
            big = kv.abs().amax(-1, keepdim=True)
            scale = torch.exp2(torch.ceil(torch.log2(torch.where(big > 0, big, 448.0) / 448)))
            kv = _to_e4m3(kv / scale) * scale
        return {"q": x[:, :, :Hq].contiguous(), "kv": kv}
    out = torch.zeros(B, R, Hq, D, dtype=torch.float64, device="cuda")
    for b in range(B):
        n, t = nodes[b] + 1, S[b]
        p = torch.arange(t if case["staged"] else t + n, device="cuda")
        e = s["kv"][s["table"][b].long()[p // case["bs"]], LAYER, :, :, p % case["bs"]]  # [keys, 2, H, E]
        if case["staged"]:
            e = torch.cat([e, s["stage"][b, :n, LAYER]])
        e = _values(e, case["kv"], D)
        q = s["q"][b, :n].double().reshape(n, Hkv, G, D)
        seen = torch.cat([torch.ones(n, t, dtype=torch.bool, device="cuda"), anc[:n, :n]], 1)
        for h in range(Hkv):
            x = torch.einsum("igd,jd->igj", q[:, h], e[:, 0, h]) / math.sqrt(D)
            x = torch.where(seen[:, None], x, -math.inf)
            out[b, :n, h * G:(h + 1) * G] = torch.einsum("igj,jd->igd", torch.softmax(x, -1), e[:, 1, h])
    return out
