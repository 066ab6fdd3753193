"""What is measured of the speculative-decoding operators: their cases, inputs, plain forms and
exact values.

A step of speculative decoding drafts a tree of tokens for every sequence, computes the target
model's logits for all of its nodes at once, keeps the nodes that the target's probabilities
accept, and leaves the cache holding those nodes only.  Node 0 is the sequence's last token
(its key and value are not in the cache before the step either); ``parents[b][i] < i`` is node
i's parent, -1 for a root.  The nodes' keys and values stand in the cache behind the ``lens[b]``
rows of the sequence, node i at row ``lens[b] + i``.  Four operators:

``attention``  every node's queries over the sequence's rows, the node's ancestors and itself
``verify``     which path of nodes the target accepts, and the token that follows it
``commit``     the accepted nodes' cache rows moved behind the sequence's rows, in every layer
``reorder``    sequences taking over other sequences' cache rows (forks of a prompt, beams)
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------ cases

def _attention(name, B, n, hq, hkv, d, length, ragged, tree, dtype):
    return dict(name=name, op="attention", B=B, n=n, hq=hq, hkv=hkv, d=d, length=length, ragged=ragged, tree=tree,
                dtype=dtype)


def _verify(name, B, n, vocab, tree, sampled, temperature, dtype):
    return dict(name=name, op="verify", B=B, n=n, vocab=vocab, tree=tree, sampled=sampled, temperature=temperature,
                dtype=dtype)


def listed():
    return [
        # one sequence of the Llama-3-8B shape in mid-answer, four drafted tokens in a row: latency
        _attention("attention chain", 1, 5, 32, 8, 128, 551, False, False, "bf16"),
        # the same model at 4 K context with a tree of 26 nodes
        _attention("attention tree 4k", 1, 26, 32, 8, 128, 4096, False, True, "bf16"),
        # the MHA model (32 KV heads) at batch 16, small trees, sequences of unlike length
        _attention("attention mha batch", 16, 13, 32, 32, 128, 1280, True, True, "bf16"),
        # few sequences with a long cache, 64-node trees: the cache's bytes count
        _attention("attention long", 4, 64, 32, 8, 128, 32768, True, True, "fp16"),
        # the widest trees: as much arithmetic as bytes; head size 64
        _attention("attention wide", 8, 256, 32, 4, 64, 4096, False, True, "bf16"),
        # four sampled tokens of one sequence against the 128256-word vocabulary: latency
        _verify("verify chain", 1, 5, 128256, False, True, 1.0, "fp32"),
        # a top-k tree (no draft probabilities), temperature below one
        _verify("verify tree", 4, 26, 65536, True, False, 0.7, "fp32"),
        # sampled trees for a whole batch; an odd vocabulary, so that rows start off 16 bytes
        _verify("verify batch", 16, 9, 128255, True, True, 0.9, "bf16"),
        # one sequence keeps a few of its nodes, every layer of the 8B shape
        dict(name="commit one", op="commit", layers=32, B=1, hkv=8, d=128, rows=1024, n=13, tree=True),
        # sixteen sequences of the MHA model keep long paths
        dict(name="commit batch", op="commit", layers=32, B=16, hkv=32, d=128, rows=192, n=64, tree=True),
        # one prompt of 39 tokens forked to four answers
        dict(name="reorder fork", op="reorder", layers=32, B=4, hkv=8, d=128, rows=256, length=39, fork=True),
        # eight beams trade places in mid-answer
        dict(name="reorder beams", op="reorder", layers=32, B=8, hkv=8, d=128, rows=1024, length=1001, fork=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "verify", "verify", "commit", "reorder"])
    if op == "attention":
        while True:
            hkv, g = rng.choice([(1, 8), (2, 2), (4, 7), (4, 8), (8, 3), (8, 4), (32, 1), (16, 2)])
            c = dict(op=op, B=_log(rng, 1, 16), n=_log(rng, 1, 256), hq=hkv * g, hkv=hkv, d=rng.choice([64, 128]),
                     length=_log(rng, 1, 32768), ragged=rng.random() < 0.5, tree=rng.random() < 0.7,
                     dtype=rng.choice(["bf16", "fp16"]))
            keys = c["B"] * hkv * (c["length"] + c["n"]) * c["d"]
            if keys <= 4 * 8 * 32768 * 128 and keys * c["n"] * g <= 8 * 4 * 4096 * 64 * 256 * 8:
                return c
    if op == "verify":
        while True:
            sampled = rng.random() < 0.5
            c = dict(op=op, B=_log(rng, 1, 32), n=_log(rng, 1, 64), vocab=_log(rng, 1000, 160000),
                     tree=rng.random() < 0.7, sampled=sampled, temperature=rng.choice([0.0, 0.6, 1.0, 1.3]),
                     dtype=rng.choice(["fp32", "bf16", "fp16"]))
            if c["B"] * c["n"] * c["vocab"] <= 16 * 9 * 128256:
                return c
    if op == "commit":
        while True:
            c = dict(op=op, layers=rng.randint(2, 40), B=_log(rng, 1, 16), hkv=rng.choice([1, 2, 4, 8, 32]),
                     d=rng.choice([64, 128]), rows=rng.randint(300, 1500), n=_log(rng, 1, 128),
                     tree=rng.random() < 0.7)
            if c["layers"] * c["B"] * c["hkv"] * c["d"] * c["rows"] <= 32 * 8 * 8 * 128 * 1024:
                return c
    while True:
        rows = _log(rng, 64, 4096)
        c = dict(op=op, layers=rng.randint(2, 40), B=rng.randint(2, 16), hkv=rng.choice([1, 2, 4, 8, 32]),
                 d=rng.choice([64, 128]), rows=rows, length=_log(rng, 16, rows), fork=rng.random() < 0.5)
        if c["layers"] * c["B"] * c["hkv"] * c["d"] * rows <= 32 * 8 * 8 * 128 * 1024:
            return c


# ----------------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda")


def _parents(g, B, n, tree):
    """Parent indices [B, n] int32: a chain, or trees a few levels deep; node 0 is the root."""
    i = torch.arange(n, device="cuda")
    if not tree:
        return (i - 1).to(torch.int32).expand(B, n).contiguous()
    p = (_rand(g, B, n) ** 1.5 * i).floor().clamp(max=n - 1)  # early nodes have more children
    p = torch.minimum(p, (i - 1).clamp(min=0).to(p.dtype))
    p[:, 0] = -1
    return p.to(torch.int32)


def _lens(g, B, length, ragged):
    if not ragged:
        return torch.full((B,), length, dtype=torch.int32, device="cuda")
    lens = (_rand(g, B) * 0.9 + 0.1).mul(length).to(torch.int32)
    lens[0] = length
    return lens


def _n_nodes(g, B, n, ragged):
    if not ragged or n < 4:
        return torch.full((B,), n, dtype=torch.int32, device="cuda")
    k = n - (_rand(g, B) * 0.3 * n).to(torch.int32)
    k[0] = n
    return k.to(torch.int32)


def _prepare_attention(c, g):
    B, n, hq, hkv, d = c["B"], c["n"], c["hq"], c["hkv"], c["d"]
    S = -(-(c["length"] + n) // 16) * 16 + 32  # rows that the cache has room for
    dt = DT[c["dtype"]]
    make = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.float32).to(dt)  # noqa: E731
    q = make(B, n, hq, d)
    kv = torch.empty(2, B, hkv, S, d, dtype=dt, device="cuda")  # one layer of the decoder's cache
    for x in range(2):
        for b in range(B):
            kv[x, b] = make(hkv, S, d)
    return dict(q=q, k=kv[0], v=kv[1], parents=_parents(g, B, n, c["tree"]), lens=_lens(g, B, c["length"], c["ragged"]),
                n_nodes=_n_nodes(g, B, n, c["ragged"]), o=torch.zeros_like(q), scale=1.0 / math.sqrt(d))


def _prepare_verify(c, g):
    B, n, V = c["B"], c["n"], c["vocab"]
    dt = DT[c["dtype"]]
    parents = _parents(g, B, n, c["tree"])
    # logits with a few likely words, as a trained model's; the draft's are the target's, blurred
    target = torch.randn(B, n, V, generator=g, device="cuda") * 2
    target += torch.where(_rand(g, B, n, V) < 3e-5, 9.0, 0.0)
    draft = target + torch.randn(B, n, V, generator=g, device="cuda") * 0.4
    target, draft = target.to(dt), draft.to(dt)
    at = parents.clamp(min=0).long()
    seq = torch.arange(B, device="cuda")[:, None]
    temp = max(c["temperature"], 0.3)
    if c["sampled"]:  # every child drawn from its parent's draft distribution
        tokens = torch.empty(B, n, dtype=torch.int64, device="cuda")
        for b in range(B):
            noise = -torch.log(-torch.log(_rand(g, n, V).clamp(1e-9, 1 - 1e-7)))
            tokens[b] = (draft[b, at[b]].float() / temp + noise).argmax(-1)
    else:  # the k-th child takes the parent's k-th likeliest word
        same = (parents[:, :, None] == parents[:, None, :]).tril(-1)
        rank = same.sum(-1)
        top = draft.float().topk(min(n, V), dim=-1).indices
        tokens = top[seq, at, rank.clamp(max=min(n, V) - 1)]
    fill = lambda t: torch.full((B,), t, dtype=torch.float32, device="cuda")  # noqa: E731
    return dict(target=target, draft=draft if c["sampled"] else None, tokens=tokens.to(torch.int32), parents=parents,
                n_nodes=_n_nodes(g, B, n, True), u=_rand(g, B, n), r=_rand(g, B),
                temperature=fill(c["temperature"]), draft_temperature=fill(temp) if c["sampled"] else None,
                path=torch.empty(B, n, dtype=torch.int32, device="cuda"),
                n_path=torch.empty(B, dtype=torch.int32, device="cuda"),
                next_token=torch.empty(B, dtype=torch.int32, device="cuda"))


def _cache(c, g):
    kv = torch.empty(c["layers"], 2, c["B"], c["hkv"], c["rows"], c["d"], dtype=torch.bfloat16, device="cuda")
    for x in kv:
        x.normal_(generator=g)
    return kv


def _prepare_commit(c, g):
    B, n = c["B"], c["n"]
    parents = _parents(g, B, n, c["tree"])
    # the path up from a late node, as long as a sequence that keeps about half of its drafts has
    node = (n - 1 - (_rand(g, B) * 0.5 * n).long()).clamp(min=0)
    keep = torch.zeros(B, n, dtype=torch.bool, device="cuda")
    seq = torch.arange(B, device="cuda")
    for _ in range(n):
        keep[seq, node] = True
        node = parents[seq, node].clamp(min=0).long()
    keep[:, 0] = True
    order = torch.argsort((~keep).to(torch.int32), dim=1, stable=True)
    n_path = keep.sum(1)
    path = torch.where(torch.arange(n, device="cuda") < n_path[:, None], order, -1)
    lens = (_rand(g, B) * (c["rows"] - n)).to(torch.int32)
    return dict(kv=_cache(c, g), path=path.to(torch.int32), n_path=n_path.to(torch.int32), lens=lens,
                new_lens=torch.empty_like(lens))


def _prepare_reorder(c, g):
    B = c["B"]
    src = torch.zeros(B, dtype=torch.int32, device="cuda")
    if not c["fork"]:
        src = (_rand(g, B) * B).to(torch.int32)  # beams: some go on, some die, some split
    lens = torch.full((B,), c["length"], dtype=torch.int32, device="cuda")
    return dict(kv=_cache(c, g), src=src, lens=lens, new_lens=torch.empty_like(lens))


def prepare(case, seed):
    make = {"attention": _prepare_attention, "verify": _prepare_verify, "commit": _prepare_commit,
            "reorder": _prepare_reorder}[case["op"]]
    return dict(make(case, _gen(seed)), op=case["op"])


# ------------------------------------------------------------------------------ plain forms

def _ancestors(parents):
    """[B, n, n] truth values: [b, i, j] whether j is i or one of its ancestors."""
    B, n = parents.shape
    seq, node = torch.arange(B, device=parents.device)[:, None], torch.arange(n, device=parents.device)
    see = (node[:, None] == node[None, :]).expand(B, n, n)
    up = parents.long()
    for _ in range(max(1, (n - 1).bit_length())):  # each round doubles the steps looked up
        above = see[seq, up.clamp(min=0)] & (up >= 0)[:, :, None]
        see = see | above
        up = torch.where(up >= 0, up[seq, up.clamp(min=0)], -1)
    return see


def _plain_attention(s):
    q, k, v = s["q"], s["k"], s["v"]
    B, n, hq, d = q.shape
    hkv, S = k.shape[1], k.shape[2]
    g = hq // hkv
    row = torch.arange(S, device=q.device)
    rel = row[None, :] - s["lens"][:, None].long()  # [B, S]: the row's node
    see = _ancestors(s["parents"])
    tree = torch.gather(see, 2, rel.clamp(0, n - 1)[:, None, :].expand(B, n, S)) & (rel < n)[:, None, :]
    see = (rel < 0)[:, None, :] | (tree & (rel >= 0)[:, None, :])  # [B, n, S]
    qg = q.float().view(B, n, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(B, hkv, g * n, d)
    sc = (qg @ k.float().transpose(-1, -2)).view(B, hkv, g, n, S) * s["scale"]
    sc = sc.masked_fill(~see[:, None, None], float("-inf"))
    p = torch.exp(sc - sc.amax(-1, keepdim=True))
    p = (p / p.sum(-1, keepdim=True)).view(B, hkv, g * n, S)
    o = (p @ v.float()).view(B, hkv, g, n, d).permute(0, 3, 1, 2, 4).reshape(B, n, hq, d).to(q.dtype)
    real = torch.arange(n, device=q.device)[None, :] < s["n_nodes"][:, None]
    s["o"].copy_(torch.where(real[:, :, None, None], o, s["o"]))
    return s["o"]


def _softmax64(x, temperature):
    """Softmax of x / temperature; at temperature 0 all on the largest value's lowest index."""
    x = x.double()
    top = x.amax(-1, keepdim=True)
    word = torch.arange(x.shape[-1], device=x.device)
    first = torch.where(x == top, word, x.shape[-1]).amin(-1, keepdim=True)
    t = temperature.double()[:, None, None]
    e = torch.exp((x - top) / torch.where(t > 0, t, 1.0))
    return torch.where(t > 0, e / e.sum(-1, keepdim=True), (word == first).double())


def _plain_verify(s):
    B, n = s["tokens"].shape
    V = s["target"].shape[-1]
    seq = torch.arange(B, device="cuda")
    p_all = _softmax64(s["target"], s["temperature"])
    q_all = _softmax64(s["draft"], s["draft_temperature"]) if s["draft"] is not None else None
    greedy = (s["temperature"] == 0)[:, None]
    word = torch.arange(V, device="cuda")
    p, cur, depth = p_all[:, 0], torch.zeros(B, dtype=torch.long, device="cuda"), torch.ones(B, dtype=torch.long, device="cuda")
    path = torch.full((B, n + 1), -1, dtype=torch.long, device="cuda")
    path[:, 0] = 0
    for c in range(1, n):  # children come in index order: every node is looked at once
        x = s["tokens"][:, c:c + 1].long()
        q = (word == x).double()
        if q_all is not None:
            q = torch.where(greedy, q, q_all[seq, cur])
        asked = (s["parents"][:, c] == cur) & (c < s["n_nodes"])
        u = torch.where(greedy[:, 0], 0.0, s["u"][:, c]).double()
        ok = asked & (u * q.gather(1, x)[:, 0] < p.gather(1, x)[:, 0])
        rest = torch.where(greedy, p, (p - q).clamp(min=0))
        left = rest.sum(-1, keepdim=True)
        p = torch.where((asked & ~ok)[:, None] & (left > 0), rest / left, p)
        p = torch.where(ok[:, None], p_all[:, c], p)
        cur = torch.where(ok, c, cur)
        path.scatter_(1, torch.where(ok, depth, n)[:, None], c)
        depth = depth + ok
    total = p.cumsum(-1)
    after = total > s["r"].double()[:, None] * total[:, -1:]
    s["next_token"].copy_(torch.where(after & (p > 0), word, V).amin(-1))
    s["path"].copy_(path[:, :n])
    s["n_path"].copy_(depth)
    return s["path"], s["n_path"], s["next_token"]


def _plain_commit(s):
    kv, path, lens = s["kv"], s["path"].long(), s["lens"].long()
    seq, j = torch.arange(path.shape[0], device="cuda")[:, None], torch.arange(path.shape[1], device="cuda")
    node = torch.where(j < s["n_path"][:, None], path, j)  # rows behind the path stay as they are
    kv[:, :, seq, :, lens[:, None] + j] = kv[:, :, seq, :, lens[:, None] + node]
    torch.add(s["lens"], s["n_path"], out=s["new_lens"])
    return kv, s["new_lens"]


def _plain_reorder(s):
    kv, src = s["kv"], s["src"].long()
    taken = s["lens"][src]
    row = torch.arange(kv.shape[4], device="cuda")
    moved = (row < taken[:, None])[None, None, :, None, :, None]
    torch.where(moved, kv[:, :, src], kv, out=kv)
    s["new_lens"].copy_(taken)
    return kv, s["new_lens"]


# ---------------------------------------------------------------------------------- one pass

def run(state):
    s, op = state, state["op"]
    if not own:
        return {"attention": _plain_attention, "verify": _plain_verify, "commit": _plain_commit,
                "reorder": _plain_reorder}[op](s)
    import persistent_megakernel_decode_04_b200 as mk
    if op == "attention":
        mk.mk_tree_attention(s["q"], s["k"], s["v"], s["o"], s["parents"], s["n_nodes"], s["lens"], s["scale"])
        return s["o"]
    if op == "verify":
        if "workspace" not in s:  # kept from step to step, as a decoding loop keeps it
            room = mk.mk_tree_verify_workspace_bytes(*s["target"].shape)
            s["workspace"] = torch.empty(room, dtype=torch.uint8, device="cuda")
        mk.mk_tree_verify(s["target"], s["draft"], s["tokens"], s["parents"], s["n_nodes"], s["u"], s["r"],
                          s["temperature"], s["draft_temperature"], s["path"], s["n_path"], s["next_token"],
                          s["workspace"])
        return s["path"], s["n_path"], s["next_token"]
    if op == "commit":
        mk.mk_cache_commit(s["kv"], s["path"], s["n_path"], s["lens"], s["new_lens"])
    else:
        mk.mk_cache_reorder(s["kv"], s["src"], s["lens"], s["new_lens"])
    return s["kv"], s["new_lens"]


def work(case):
    c, op = case, case["op"]
    if op == "attention":
        # sequences of unlike length are 0.1 to 1 times the longest
        keys = c["length"] * (1 + (c["B"] - 1) * 0.55) if c["ragged"] else c["length"] * c["B"]
        rows = keys + c["B"] * c["n"]
        return {"bytes": 2 * (2 * rows * c["hkv"] * c["d"] + 2 * c["B"] * c["n"] * c["hq"] * c["d"]),
                "flops": 4 * rows * c["n"] * c["hq"] * c["d"]}
    if op == "verify":
        # every node's target row; the draft rows of nodes with children: all but the last of a
        # chain, about half of a tree's
        draft = 0 if not c["sampled"] or c["temperature"] == 0 else c["n"] - 1 if not c["tree"] else c["n"] / 2
        values = c["B"] * c["vocab"] * (c["n"] + draft)
        return {"bytes": values * (4 if c["dtype"] == "fp32" else 2), "flops": 4 * values}
    row = c["layers"] * 2 * c["hkv"] * c["d"] * 2
    if op == "commit":
        # half of a chain is kept and stays where it is; a tree's path is a few rows, read and written
        kept = 0.75 * c["n"] if not c["tree"] else 1.5 * math.log(c["n"] + 1)
        return {"bytes": c["B"] * (2 * row * kept + 8 * c["n"]), "flops": 0}
    if c["fork"]:  # one sequence read, all others written
        return {"bytes": row * c["length"] * c["B"], "flops": 0}
    # about 1 - 1/e of the sequences are read, and nearly all of them written
    return {"bytes": row * c["length"] * c["B"] * 1.55, "flops": 0}


# ------------------------------------------------------------------------------ exact values

def exact(case, seed):
    """Attention sequence by sequence in 64 bits, each node's rows found by walking up to the
    root.  What the other operators return are whole numbers and copied values."""
    if case["op"] != "attention":
        return None
    s = prepare(case, seed)
    parents, lens, n_nodes = s["parents"].tolist(), s["lens"].tolist(), s["n_nodes"].tolist()
    B, n, hq, d = s["q"].shape
    g = hq // s["k"].shape[1]
    out = s["o"].double()
    for b in range(B):
        total = lens[b] + n
        hidden = torch.ones(n, n, dtype=torch.bool)
        for i in range(n):
            j = i
            while j >= 0:
                hidden[i, j] = False
                j = parents[b][j]
        hidden = hidden.cuda()
        for h in range(hq):
            k, v = s["k"][b, h // g, :total].double(), s["v"][b, h // g, :total].double()
            x = torch.mm(s["q"][b, :, h].double(), k.t()) * s["scale"]
            x[:, lens[b]:].masked_fill_(hidden, -math.inf)
            out[b, :n_nodes[b], h] = torch.mm(torch.softmax(x, dim=1), v)[:n_nodes[b]]
    return out
