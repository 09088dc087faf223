"""Attention that shares prefixes and shapes its scores, as cases to time and compare.

Three operators next to the attention of a verify pass over the paged cache:

  groups   block tables and lengths -> which neighbouring requests hold the same leading blocks
  shared   the attention of a batch whose groups share a prefix: the prefix's keys and values are
           read once for all of a group's rows
  forms    the attention with capped scores (c tanh(s / c)), a bias that grows with the distance
           (one slope a head), a window of the nearest positions, alone or together

`own = False` runs them in elementary torch operations in 32 bits; `own = True` through the
package's public calls.  Sizes are those of the repository's own workloads: 256 requests of 4
drafts whose groups of 4 share 1024 tokens, 28 heads over 4 KV heads x d128; 32 heads over 8 KV
heads x d128 in bf16 or 8 bits; 4 heads x d64 fp32; blocks of 16; trees of the named shapes.
"""

import math
import random

import numpy as np
import torch

own = False

E4M3_TAIL = 16  # bytes after an entry's codes: its fp32 scale, then zeros
LEAST = 128     # positions below which neighbours are not grouped


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
    r = random.Random(int(arg))
    return [r.randrange(i) for i in range(1, int(arg) + 1)]


def ancestors(par):
    """(bits, depth) of one tree."""
    n = len(par) + 1
    a, depth = np.zeros((n, n), bool), np.zeros(n, np.int64)
    a[0, 0] = True
    for i in range(1, n):
        a[i] = a[par[i - 1]]
        a[i, i] = True
        depth[i] = depth[par[i - 1]] + 1
    return a, depth


def lengths(case):
    """The requests' cached lengths: a shared prefix and [lo, hi] positions of each one's own."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    s = [lo + (hi - lo) * b // max(1, B - 1) for b in range(B)] if B > 1 else [hi]
    random.Random(B * 7919 + hi).shuffle(s)
    return [case["prefix"] + x for x in s]


def common_blocks(case, seed=None):
    """For each request, how many of its leading blocks are its left neighbour's; with a seed,
    requests left their group's prompt at any point."""
    B, g, bs = case["B"], case["group"], case["bs"]
    S = lengths(case)
    r = random.Random(seed)
    most = [min(case["prefix"], S[b - 1], S[b]) // bs if b % g else 0 for b in range(B)]
    return most if seed is None else [r.randint(0, m) for m in most]


def grouping(case):
    """(shared positions [B], members [B]) by the definition, on the host: neighbours belong
    together where at least LEAST positions' blocks are the same; a group shares the least."""
    B, bs, c = case["B"], case["bs"], common_blocks(case)
    length, members, b = [0] * B, [0] * B, 0
    while b < B:
        e = b + 1
        while e < B and c[e] > 0 and c[e] * bs >= LEAST:
            e += 1
        if e - b > 1:
            members[b] = e - b
            length[b:e] = [bs * min(c[b + 1:e])] * (e - b)
        b = e
    return length, members


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
def _attention(name, op, B, tree, *, lo=0, hi, prefix=0, group=1, heads=(32, 8, 128), kv="bf16", staged=True, ragged=False,
               bs=16, cap=0.0, slopes=False, window=0):
    return dict(name=name, op=op, B=B, tree=tree, lo=lo, hi=hi, prefix=prefix, group=group, Hq=heads[0], Hkv=heads[1],
                D=heads[2], kv=kv, staged=staged, ragged=ragged, bs=bs, cap=cap, slopes=slopes, window=window)


def listed():
    return [
        # a few requests that left one prompt, looked over once a step
        dict(name="groups_b4", op="groups", B=4, prefix=1024, group=4, lo=0, hi=31, bs=16),
        # a large batch whose forks left their common prompt at different points
        dict(name="groups_b256", op="groups", B=256, prefix=8192, group=16, lo=0, hi=500, bs=16),
        # four samples of one prompt, a token each: the smallest sharing step
        _attention("shared_token_b4", "shared", 4, "chain:0", lo=1, hi=60, prefix=777, group=4, staged=False),
        # 256 requests of four drafts, groups of four over 1024 shared tokens and a few of their own
        _attention("shared_chain_b256", "shared", 256, "chain:4", hi=31, prefix=1024, group=4, heads=(28, 4, 128)),
        # one instruction of 2048 tokens before all of a batch's own prompts
        _attention("shared_token_b64", "shared", 64, "chain:0", lo=128, hi=4096, prefix=2048, group=64, staged=False),
        # trees below documents that sixteen requests each ask about, cached in 8 bits
        _attention("shared_tree_e4m3", "shared", 64, "binary:3", lo=5, hi=700, prefix=8192, group=16, kv="e4m3", ragged=True),
        # the same way with heads that weigh by distance
        _attention("shared_slopes_b64", "shared", 64, "binary:2", lo=1, hi=300, prefix=4100, group=8, slopes=True),
        # one request's smallest step: fp32 heads of 64, five drafts in a chain, 32 cached tokens
        _attention("cap_fp32_b1", "forms", 1, "chain:5", lo=32, hi=32, heads=(4, 4, 64), kv="fp32", cap=30.0),
        # a serving batch of trees with capped scores
        _attention("cap_tree_b64", "forms", 64, "binary:3", lo=128, hi=8192, cap=50.0),
        # the same batch over an 8-bit cache, heads that weigh by distance
        _attention("slopes_tree_e4m3", "forms", 64, "binary:3", lo=128, hi=8192, kv="e4m3", slopes=True),
        # layers that see the nearest 1024 positions, single tokens
        _attention("window_token_b64", "forms", 64, "chain:0", lo=128, hi=8192, staged=False, window=1024, cap=50.0),
        # prompts of such a layer
        _attention("window_prompt_b4", "forms", 4, "chain:2040", lo=0, hi=2048, staged=False, ragged=True, window=1024),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _tree(rng, most):
    kind = rng.choice(["chain", "binary", "random"])
    if kind == "binary":
        return "binary:%d" % rng.randint(1, max(1, int(math.log2(most + 2)) - 1))
    return "%s:%d" % (kind, rng.randint(0, most) if kind == "chain" else _log(rng, 1, most))


def _drawn(rng):
    op = rng.choice(["groups", "shared", "shared", "shared", "forms", "forms", "forms"])
    bs = rng.choice([16, 16, 16, 32, 64, 8])
    if op == "groups":
        B = _log(rng, 4, 256)
        return dict(op=op, B=B, prefix=_log(rng, 1024, 8192), group=_log(rng, 4, B), lo=0, hi=_log(rng, 1, 500), bs=bs)
    heads = rng.choice([(32, 8, 128), (28, 4, 128), (8, 8, 64), (16, 2, 64), (32, 8, 128)])
    kv = rng.choice(["bf16", "e4m3"])
    forms = dict(cap=rng.choice([0.0, 30.0, 50.0, rng.uniform(5.0, 100.0)]), slopes=rng.random() < 0.4,
                 window=rng.choice([0, 0, _log(rng, 1, 4096)]))
    tree = "chain:0" if rng.random() < 0.3 else _tree(rng, 14)
    place = dict(staged=rng.random() < 0.6, ragged=rng.random() < 0.4, bs=bs)
    if op == "shared":
        B, hi = _log(rng, 2, 256), _log(rng, 1, 8192)
        if rng.random() < 0.7:
            forms = {}
        case = _attention("", op, B, tree, lo=rng.randint(0, hi), hi=hi, prefix=_log(rng, 100, 8192), group=_log(rng, 1, B),
                          heads=heads, kv=kv, **place, **forms)
    elif rng.random() < 0.2:  # the fp32 cache is the small configuration's
        B, hi = _log(rng, 1, 8), _log(rng, 1, 512)
        case = _attention("", op, B, tree, lo=rng.randint(0, hi), hi=hi, heads=(4, 4, 64), kv="fp32", **place, **forms)
    else:
        B, hi = _log(rng, 1, 64), _log(rng, 1, 65536)
        if rng.random() < 0.3:
            tree = rng.choice(["random:%d", "chain:%d"]) % _log(rng, 15, 2040)
        case = _attention("", op, B, tree, lo=rng.randint(0, hi), hi=hi, heads=heads, kv=kv, **place, **forms)
    del case["name"]
    return case


def _rows(case):
    return case["B"] * len(tree_parents(case["tree"]) + [0])


def draw(rng):
    """A case of the listed ones' ranges that costs no more than the largest of them."""
    most = [work(c) for c in listed()]
    while True:
        case = _drawn(rng)
        # trees past a few hundred nodes are chains (prompts): a mask of any other takes R^2 words
        if case["op"] != "groups" and (_rows(case) > 8200 or case["tree"].startswith("random") and _rows(case) // case["B"] > 300):
            continue
        if case["op"] == "forms" and case["B"] * case["hi"] > 64 * 8192:
            continue
        w = work(case)
        if all(w[k] <= max(x[k] for x in most) for k in w):
            return case


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


def _table(case, gen, more, seed=None):
    """Block tables over a pool whose blocks are handed out in random order, leading blocks taken
    over from the left neighbour where requests share them; -1 past the last."""
    bs, S = case["bs"], lengths(case)
    n = [-(-(s + more) // bs) for s in S]
    c = common_blocks(case, seed)
    total, width = sum(n) - sum(c), max(1, max(n))
    order = torch.randperm(max(1, total), generator=gen, device=gen.device).cpu().numpy().astype(np.int32)
    table, at = np.full((case["B"], width), -1, np.int32), 0
    for b, m in enumerate(n):
        table[b, :c[b]] = table[b - 1, :c[b]]
        table[b, c[b]:m] = order[at:at + m - c[b]]
        at += m - c[b]
    return torch.tensor(table, device="cuda"), max(1, total)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _pack(bits):
    """[..., n] truth values -> [..., ceil(n / 32)] int32 words, bit j of word w standing for 32 w + j."""
    n = bits.shape[-1]
    bits = torch.nn.functional.pad(bits, (0, -n % 32)).reshape(*bits.shape[:-1], -1, 32)
    words = (bits.long() << torch.arange(32, device=bits.device)).sum(-1)
    return torch.where(words >= 1 << 31, words - (1 << 32), words).int()


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    B = case["B"]
    s = dict(case=case, B=B, seq_len=_ints(lengths(case)))
    if case["op"] == "groups":
        s["table"], _ = _table(case, gen, 1, seed)
        return s
    par = tree_parents(case["tree"])
    R = len(par) + 1
    bits, depth = ancestors(par)
    n = torch.tensor(nodes_of(case), device="cuda")
    alive = torch.arange(R, device="cuda") <= n[:, None]
    s.update(R=R, n_nodes=n.int())
    s["mask"] = _pack(torch.tensor(bits, device="cuda") & alive[:, :, None]).contiguous()
    s["depth"] = (torch.tensor(depth, device="cuda") * alive).int().contiguous()
    Hq, Hkv, D, kv = case["Hq"], case["Hkv"], case["D"], case["kv"]
    dt = torch.float32 if kv == "fp32" else torch.bfloat16
    s["table"], blocks = _table(case, gen, 0 if case["staged"] else R)
    s["kv"] = _entries((blocks, LAYERS, 2, Hkv, case["bs"]), kv, D, gen)
    s["stage"] = _entries((B, R, LAYERS, 2, Hkv), kv, D, gen) if case["staged"] else None
    s["q"] = torch.randn(B, R, Hq, D, generator=gen, device="cuda", dtype=dt)
    s["out"] = torch.empty_like(s["q"])
    # every head its slope, from a half down to 2^-8 for 8 heads
    s["slopes"] = torch.exp2(-8.0 * torch.arange(1, Hq + 1, device="cuda") / Hq).float() if case["slopes"] else None
    s["groups"] = None
    if case["op"] == "shared":  # made once a step, for all layers
        length, members = grouping(case)
        s["groups"] = dict(length=_ints(length), members=_ints(members))
    return s


# --------------------------------------------------------------------------- #
# plain forms: elementary operations in 32 bits
# --------------------------------------------------------------------------- #
def _plain_groups(s):
    bs, t, S = s["case"]["bs"], s["table"], s["seq_len"]
    B, width = t.shape
    j = torch.arange(width, device="cuda")
    most = torch.minimum(S, S.roll(1)) // bs
    same = (t == t.roll(1, 0)) & (t >= 0) & (j < most[:, None])
    c = same.int().cumprod(1).sum(1) * bs
    c[0] = 0
    joined = (c > 0) & (c >= LEAST)
    group = (~joined).int().cumsum(0) - 1
    least = torch.full((B,), 1 << 30, dtype=c.dtype, device="cuda").scatter_reduce(0, group, torch.where(joined, c, 1 << 30), "amin")
    count = torch.zeros(B, dtype=torch.int64, device="cuda").scatter_add(0, group, torch.ones_like(group))
    many = count[group] > 1
    return {"length": torch.where(many, least[group], 0).int(),
            "members": torch.where(many & ~joined, count[group], 0).int()}


def _unpack(words, n):
    return ((words.unsqueeze(-1) >> torch.arange(32, device=words.device, dtype=torch.int32)) & 1).flatten(-2)[..., :n].bool()


def _decode(x, kv, D):
    if kv != "e4m3":
        return x.float()
    scale = x[..., D:D + 4].contiguous().view(torch.float32)
    return x[..., :D].view(torch.float8_e4m3fn).float() * scale


def _plain_attention(s, b0, b1):
    c, R, D, bs = s["case"], s["R"], s["case"]["D"], s["case"]["bs"]
    H, G, B = c["Hkv"], c["Hq"] // c["Hkv"], b1 - b0
    pages = _decode(s["kv"][s["table"][b0:b1].long().clamp(min=0), LAYER], c["kv"], D)  # [B, m, 2, H, bs, D]
    kv = pages.permute(2, 0, 3, 1, 4, 5).reshape(2, B, H, -1, D)
    S, n, depth = s["seq_len"][b0:b1, None], s["n_nodes"][b0:b1, None], s["depth"][b0:b1]
    at = torch.arange(kv.shape[3], device="cuda") - S  # 0 is the pending token
    live = torch.arange(R, device="cuda") <= n
    bits = _unpack(s["mask"][b0:b1], R) & live[:, None]
    if c["staged"]:
        kv = torch.cat([kv, _decode(s["stage"][b0:b1, :, LAYER], c["kv"], D).permute(2, 0, 3, 1, 4)], 3)
        seen = torch.cat([(at < 0)[:, None].expand(B, R, -1), bits], 2)
        place = torch.cat([at, depth], 1)
    else:
        entry = at.clamp(0, R - 1).long()
        seen = (at < 0)[:, None] | ((at < R)[:, None] & bits.gather(2, entry[:, None].expand(B, R, -1)))
        place = torch.where(at < 0, at, depth.gather(1, entry))
    far = (depth[:, :, None] - place[:, None]).abs()  # [B, R, keys]
    if c["window"]:
        seen = seen & (far < c["window"])
    q = s["q"][b0:b1].float().reshape(B, R, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, R * G, D)
    x = (q @ kv[0].transpose(2, 3) / math.sqrt(D)).reshape(B, H, R, G, -1)
    if c["cap"]:
        x = c["cap"] * torch.tanh(x / c["cap"])
    if c["slopes"]:
        x = x - s["slopes"].reshape(H, 1, G, 1) * far[:, None, :, None].float()
    x = x.masked_fill(~seen[:, None, :, None], -math.inf)
    x = x - x.amax(-1, keepdim=True).clamp(min=-3e38)
    x = x.exp_().reshape(B, H, R * G, -1)
    o = (x @ kv[1]) / x.sum(-1, keepdim=True).clamp(min=1e-30)
    o = o.reshape(B, H, R, G, D).permute(0, 2, 1, 3, 4).reshape(B, R, c["Hq"], D)
    return (o * live[:, :, None, None]).to(s["q"].dtype)


def _plain(s):
    if s["case"]["op"] == "groups":
        return _plain_groups(s)
    c = s["case"]
    # as many requests at a time as a few GB of scores and pages allow
    keys = s["table"].shape[1] * c["bs"] + s["R"]
    per = max(1, (1 << 30) // (keys * max(s["R"] * c["Hq"], 4 * c["Hkv"] * c["D"])))
    return torch.cat([_plain_attention(s, b, min(s["B"], b + per)) for b in range(0, s["B"], per)])


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
    if c["op"] == "groups":
        return ver.prefix_groups(s["table"], s["seq_len"], c["bs"], least=LEAST)
    return ver.tree_attention(s["q"], s["kv"], s["table"], s["seq_len"], layer=LAYER, stage=s["stage"], mask=s["mask"],
                              n_nodes=s["n_nodes"], out=s["out"], depth=s["depth"], softcap=c["cap"] or None,
                              slopes=s["slopes"], window=c["window"] or None, groups=s["groups"])


def run(state):
    return _own(state) if own else _plain(state)


# --------------------------------------------------------------------------- #
# what a pass cannot do without
# --------------------------------------------------------------------------- #
def work(case):
    S = lengths(case)
    if case["op"] == "groups":
        common = [min(x + 1, a // case["bs"], b // case["bs"]) for x, a, b in zip(common_blocks(case)[1:], S, S[1:])]
        return {"bytes": 4 * (3 * case["B"] + 2 * sum(common)), "flops": 0}
    a, depth = ancestors(tree_parents(case["tree"]))
    nodes, W, D = nodes_of(case), case["window"], case["D"]
    Hq, Hkv, eb = case["Hq"], case["Hkv"], 4 if case["kv"] == "fp32" else 2
    rows = sum(n + 1 for n in nodes)
    near = a & (depth[:, None] - depth[None] < W) if W else a
    pairs = keys = 0
    for s, n in zip(S, nodes):
        d = depth[:n + 1]
        pairs += int(near[:n + 1].sum()) + int(np.clip(W - 1 - d, 0, s).sum() if W else s * (n + 1))
        keys += n + 1 + (min(s, W - 1) if W else s)
    if case["op"] == "shared" and not W:  # a group's prefix is read once
        length, members = grouping(case)
        keys -= sum((m - 1) * x for x, m in zip(length, members) if m)
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


def exact(case, seed):
    if case["op"] == "groups":
        return None  # whole numbers: the plain form's have to be met
    s = prepare(case, seed)
    B, R, nodes, S = s["B"], s["R"], nodes_of(case), lengths(case)
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    G = Hq // Hkv
    anc, depth = (torch.tensor(x, device="cuda") for x in ancestors(tree_parents(case["tree"])))
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
        where = torch.cat([torch.arange(t, device="cuda"), t + depth[:n]])  # positions of keys
        apart = torch.abs(t + depth[:n, None] - where[None])
        if case["window"]:
            seen &= apart < case["window"]
        for h in range(Hkv):
            x = torch.einsum("igd,jd->igj", q[:, h], e[:, 0, h]) / math.sqrt(D)
            if case["cap"]:
                x = case["cap"] * torch.tanh(x / case["cap"])
            if case["slopes"]:
                x = x - s["slopes"][h * G:(h + 1) * G].double()[None, :, None] * apart[:, None].double()
            x = torch.where(seen[:, None], x, -math.inf)
            out[b, :n, h * G:(h + 1) * G] = torch.einsum("igj,jd->igd", torch.softmax(x, -1), e[:, 1, h])
    return out
