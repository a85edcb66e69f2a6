"""Timed cases of the operators around a drafted token tree.

Four operators, each in its plain form (elementary torch operations in 32
bits, rounded once at the end) and through the library's entry points:

  tree_attention  attention of a tree's (or chain's) query rows over a paged
                  key/value cache and their own ancestors
  append_nodes    norms of queries and keys per head, the rotation by each
                  node's position, and the write of keys and values into the
                  cache
  keep_path       moves the accepted path's cache rows to the places they
                  keep
  process_logits  penalties for repeated tokens, biases and grammar masks on
                  the logits of every node

`own` selects the side: False runs the plain forms, True the library.
"""

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # one user, one token at a time, a short conversation: latency
        dict(name="attn-one-token", op="attn", dtype="bf16", B=1, N=1, nlo=1, Hq=32, Hkv=8, D=128,
             page=16, lo=1999, hi=1999, chain=True),
        # a served batch, a tree of 32 candidates each, ragged contexts
        dict(name="attn-tree-batch", op="attn", dtype="bf16", B=32, N=32, nlo=9, Hq=32, Hkv=8,
             D=128, page=64, lo=97, hi=4093, chain=False),
        # few users with long documents, K = 4 drafts in a chain
        dict(name="attn-chain-long", op="attn", dtype="bf16", B=8, N=5, nlo=2, Hq=32, Hkv=8,
             D=128, page=64, lo=16111, hi=32749, chain=True),
        # the widest trees: 64 candidates, eight query heads to each key head
        dict(name="attn-tree-wide", op="attn", dtype="f16", B=32, N=64, nlo=64, Hq=64, Hkv=8,
             D=128, page=32, lo=4001, hi=8111, chain=False),
        # one user's chain of K = 4 drafts, norms and half layout
        dict(name="append-one-chain", op="append", dtype="bf16", B=1, N=5, nlo=5, Hq=32, Hkv=8,
             D=128, page=16, lo=1999, hi=1999, chain=True, rot=128, interleaved=False, norm=True),
        # a served batch of trees, interleaved pairs on half of each head, no norm
        dict(name="append-tree-batch", op="append", dtype="f16", B=32, N=32, nlo=9, Hq=32, Hkv=8,
             D=128, page=64, lo=97, hi=4093, chain=False, rot=64, interleaved=True, norm=False),
        # a full machine: 256 trees of 32 nodes at far positions
        dict(name="append-tree-full", op="append", dtype="bf16", B=256, N=32, nlo=17, Hq=64, Hkv=8,
             D=128, page=64, lo=60013, hi=131009, chain=False, rot=128, interleaved=False,
             norm=True),
        # one user's tree, one layer
        dict(name="keep-one-layer", op="keep", dtype="bf16", B=1, N=32, nlo=32, Hkv=8, D=128,
             page=16, lo=1999, hi=1999, layers=1, deep=4),
        # a served batch, every layer of the model in one call
        dict(name="keep-all-layers", op="keep", dtype="bf16", B=128, N=64, nlo=33, Hkv=8, D=128,
             page=64, lo=131, hi=509, layers=16, deep=6),
        # one user's K = 4 drafts before verification: penalties and a bias, f32 logits
        dict(name="logits-one-chain", op="logits", dtype="f32", B=1, N=5, nlo=5, V=128256, chain=True,
             hist=1024, lo=700, hi=700, nbias=16, mask=False),
        # the DeepSeek-class draft step with penalties and a grammar: 512 requests, K = 1
        dict(name="logits-batch-masked", op="logits", dtype="bf16", B=512, N=2, nlo=1, V=129280,
             chain=True, hist=4096, lo=33, hi=4001, nbias=0, mask=True),
        # 32 trees of 32 nodes, every node under its own path's penalties
        dict(name="logits-tree-batch", op="logits", dtype="bf16", B=32, N=32, nlo=9, V=128256,
             chain=False, hist=8192, lo=500, hi=8100, nbias=64, mask=True),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["attn", "attn", "append", "keep", "logits"])
    B, N = _log(rng, 1, 64), _log(rng, 1, 64)
    page = rng.choice([1, 8, 16, 24, 32, 64, 100, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    D = rng.choice([64, 64, 80, 96, 128, 128, 128])
    dtype = rng.choice(["bf16", "f16"])
    nlo = rng.choice([N, max(1, N // 3)])
    chain = rng.random() < 0.4
    if op == "attn":
        G = rng.choice([1, 2, 3, 4, 5, 7, 8])
        most = min(32749, 32 * 8111 * 8 * 128 // (B * Hkv * 128), 32 * 64 * 64 * 8111 // (B * N * Hkv * G))
        hi = min(_log(rng, 1, 32749), most)
        return dict(op=op, dtype=dtype, B=B, N=N, nlo=nlo, Hq=Hkv * G, Hkv=Hkv, D=D, page=page,
                    lo=rng.choice([hi, hi // 2, hi // 50]), hi=hi, chain=chain)
    if op == "append":
        hi = min(_log(rng, 1, 131009), 32 * 131009 // B)
        return dict(op=op, dtype=dtype, B=B, N=N, nlo=nlo, Hq=Hkv * rng.choice([1, 2, 4, 8]), Hkv=Hkv,
                    D=D, page=page, lo=hi // 3, hi=hi, chain=chain, rot=rng.choice([D, D // 2, 0]),
                    interleaved=rng.random() < 0.5, norm=rng.random() < 0.6)
    if op == "keep":
        return dict(op=op, dtype=dtype, B=B, N=N, nlo=nlo, Hkv=Hkv, D=D, page=page,
                    lo=rng.randint(0, 100), hi=rng.randint(100, 509), layers=rng.randint(1, 16),
                    deep=rng.randint(0, 8))
    N = min(N, 32)
    B = min(B, 32)
    hist = _log(rng, 8, 8192)
    return dict(op=op, dtype=rng.choice(["bf16", "f32"]), B=B, N=N, nlo=min(nlo, N),
                V=rng.choice([1024, 32003, 50000, 128256, 129280]) if B * N < 512 else 50000,
                chain=chain, hist=hist, lo=rng.randint(0, hist // 2), hi=rng.randint(hist // 2, hist),
                nbias=rng.choice([0, 5, 64]), mask=rng.random() < 0.5)


def _spread(lo, hi, B):
    """B whole numbers from lo to hi, evenly: the case's lengths, whatever the seed."""
    return np.rint(np.linspace(lo, hi, B)).astype(np.int64) if B > 1 else np.array([hi])


def _trees(rs, B, N):
    parents = np.full((B, N), -1, np.int32)
    for i in range(1, N):
        parents[:, i] = rs.randint(0, i, B)
    return parents


def _put(a, dtype=None):
    return torch.from_numpy(np.ascontiguousarray(a, dtype)).cuda()


def prepare(case, seed):
    c, rs = dict(case), np.random.RandomState(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[c["dtype"]]
    B, N = c["B"], c["N"]

    def normal(*shape, scale=1.0, dtype=dt):
        return torch.randn(*shape, generator=gen, device="cuda").mul_(scale).to(dtype)

    # lengths are the case's own (work() counts them); the seed says whose is which
    lens = rs.permutation(_spread(c["lo"], c["hi"], B))
    nodes = rs.permutation(_spread(c["nlo"], N, B))
    s = dict(case=c, n_nodes=_put(nodes, np.int32), status=torch.zeros(B, dtype=torch.int32, device="cuda"))
    if c["op"] in ("attn", "append", "keep"):
        P = -(-(c["hi"] + N) // c["page"])
        if c["op"] == "append":  # only the pages that the nodes fall in are this call's own
            first = lens // c["page"]
            own_pages = (lens + N - 1) // c["page"] - first + 1
            table = np.zeros((B, P), np.int64)
            ids = rs.permutation(int(own_pages.sum())) + 1
            at = np.cumsum(own_pages) - own_pages
            for b in range(B):
                table[b, first[b]:first[b] + own_pages[b]] = ids[at[b]:at[b] + own_pages[b]]
            pages = int(own_pages.sum()) + 1
        else:
            table, pages = rs.permutation(B * P).reshape(B, P), B * P
        Hkv, D = c["Hkv"], c["D"]
        s.update(page_table=_put(table, np.int32), cache_lens=_put(lens, np.int32))
        layers = [c["layers"]] if c["op"] == "keep" else []
        s["k_cache"] = torch.empty(*layers, pages, c["page"], Hkv, D, dtype=dt, device="cuda")
        s["v_cache"] = torch.empty_like(s["k_cache"])
        for one in ("k_cache", "v_cache"):
            for part in (s[one] if layers else [s[one]]):
                part.copy_(normal(*part.shape))
    if c["op"] in ("attn", "append"):
        s["parents"] = None if c["chain"] else _put(_trees(rs, B, N), np.int32)
        Hq = c["Hq"]
        # the projection's output, queries, keys and values side by side in one row
        qkv = normal(B, N, (Hq + 2 * Hkv) * D)
        q, k, v = qkv.split([Hq * D, Hkv * D, Hkv * D], dim=-1)
        s.update(q=q.unflatten(-1, (Hq, D)), k=k.unflatten(-1, (Hkv, D)), v=v.unflatten(-1, (Hkv, D)),
                 out=torch.zeros(B, N, Hq, D, dtype=dt, device="cuda"))
    if c["op"] == "append":
        rot = c["rot"] // 2 * 2
        s["inv_freq"] = _put(500000.0 ** (-np.arange(0, rot, 2) / max(rot, 1)), np.float32) if rot else None
        s["q_weight"] = (1 + normal(D, scale=0.1, dtype=torch.float32)).to(dt) if c["norm"] else None
        s["k_weight"] = (1 + normal(D, scale=0.1, dtype=torch.float32)).to(dt) if c["norm"] else None
    if c["op"] == "keep":
        path, accepted = np.full((B, N), -1, np.int32), np.zeros(B, np.int32)
        for b in range(B):
            # sources behind the destinations, so that a second pass moves the same rows again
            A = min(int(rs.randint(0, c["deep"] + 1)), (int(nodes[b]) - 1) // 2)
            path[b, 0] = 0
            path[b, 1:A + 1] = np.sort(rs.choice(np.arange(A + 1, nodes[b]), A, replace=False))
            accepted[b] = A
        s.update(path_nodes=_put(path), accepted_len=_put(accepted),
                 new_lens=torch.zeros(B, dtype=torch.int32, device="cuda"))
    if c["op"] == "logits":
        V, L = c["V"], c["hist"]
        s["logits"] = normal(B, N, V, scale=3.0)
        # word frequencies of a text: few tokens often, most hardly ever
        zipf = np.minimum((V ** rs.random_sample((B, L))).astype(np.int64), V) - 1
        perm = rs.permutation(V)
        s["history"] = _put(perm[zipf], np.int32)
        s["seq_lens"] = _put(lens, np.int32)
        s["prompt_lens"] = _put((lens * rs.random_sample(B)).astype(np.int64), np.int32)
        tokens = perm[np.minimum((V ** rs.random_sample((B, N))).astype(np.int64), V) - 1]
        s["tokens"] = _put(tokens, np.int32)
        s["drafts"] = _put(tokens[:, 1:], np.int32)  # a chain's, as the verification takes them
        s["parents"] = None if c["chain"] else _put(_trees(rs, B, N), np.int32)
        s["repetition"] = _put(rs.uniform(1.0, 1.3, B), np.float32)
        s["frequency"] = _put(rs.uniform(0.0, 0.5, B), np.float32)
        s["presence"] = _put(rs.uniform(0.0, 0.5, B), np.float32)
        s["bias_tokens"] = s["bias_values"] = s["allowed"] = None
        if c["nbias"]:
            pick = np.argsort(rs.random_sample((B, min(V, 20 * c["nbias"]))), axis=1)[:, :c["nbias"]]
            s["bias_tokens"] = _put(perm[pick * (V // min(V, 20 * c["nbias"]))], np.int32)
            s["bias_values"] = _put(rs.uniform(-5, 5, pick.shape), np.float32)
        if c["mask"]:
            # a grammar's bits: between everything and next to nothing, by node
            W = -(-V // 32)
            bits = torch.randint(-2 ** 31, 2 ** 31 - 1, (B, N, W), generator=gen, device="cuda")
            bits &= torch.randint(-2 ** 31, 2 ** 31 - 1, (B, N, W), generator=gen, device="cuda")
            dense = torch.rand(B, N, W, generator=gen, device="cuda")
            keep = torch.rand(B, N, 1, generator=gen, device="cuda")
            s["allowed"] = torch.where(dense < keep * keep, bits, bits * 0).to(torch.int32)
        s["out"] = torch.zeros(B, N, V, dtype=dt, device="cuda")
    return s


def _ancestors(s):
    """[B, N, N] of truth values: node i sees node j (its ancestors and itself)."""
    c = s["case"]
    N = c["N"]
    if s["parents"] is None:
        up = torch.ones(N, N, device="cuda").tril()[None].expand(c["B"], N, N)
    else:
        at = torch.arange(N, device="cuda")
        up = (s["parents"][:, :, None] == at).float() + torch.eye(N, device="cuda")
        up = torch.matrix_power(up, 64)
    return up > 0


def _rows(cache, table):
    """The cache's rows in each request's order, [B, P * page, Hkv, D]."""
    return cache[table.long()].flatten(1, 2)


def _plain_attn(s):
    c = s["case"]
    B, N, Hq, Hkv, D = (c[k] for k in ("B", "N", "Hq", "Hkv", "D"))
    G = Hq // Hkv
    k = _rows(s["k_cache"], s["page_table"]).float()
    q = s["q"].float().reshape(B, N, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, N * G, D)
    scores = (q @ k.permute(0, 2, 3, 1)).mul_(D ** -0.5)
    del k
    L = scores.shape[-1]
    behind = torch.arange(L, device="cuda")[None] - s["cache_lens"].long()[:, None]
    drafted = (behind >= 0) & (behind < s["n_nodes"].long()[:, None])
    tree = _ancestors(s).gather(2, behind.clamp(0, N - 1)[:, None].expand(B, N, L))
    seen = (behind < 0)[:, None] | (tree & drafted[:, None])
    scores.view(B, Hkv, N, G, L).masked_fill_(~seen[:, None, :, None], float("-inf"))
    scores -= scores.amax(-1, keepdim=True)
    scores.exp_()
    scores /= scores.sum(-1, keepdim=True)
    v = _rows(s["v_cache"], s["page_table"]).float()
    o = (scores @ v.permute(0, 2, 1, 3)).reshape(B, Hkv, N, G, D).permute(0, 2, 1, 3, 4).reshape(B, N, Hq, D)
    real = torch.arange(N, device="cuda")[None] < s["n_nodes"][:, None]
    s["out"].copy_(torch.where(real[:, :, None, None], o, 0.0))
    return s["out"], s["status"]


def _plain_append(s):
    c = s["case"]
    B, N, D = c["B"], c["N"], c["D"]
    real = torch.arange(N, device="cuda")[None] < s["n_nodes"][:, None]
    depth = _ancestors(s).sum(-1) - 1
    pos = s["cache_lens"].long()[:, None] + depth

    def turn(x, weight):
        x = x.float()
        if weight is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * weight.float()
        if s["inv_freq"] is None:
            return x
        angle = pos[:, :, None, None].double() * s["inv_freq"].double()
        cos, sin = angle.cos().float(), angle.sin().float()
        rot = 2 * s["inv_freq"].numel()
        if c["interleaved"]:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            both = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = x[..., :rot // 2], x[..., rot // 2:rot]
            both = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([both, x[..., rot:]], -1)

    s["out"].copy_(torch.where(real[:, :, None, None], turn(s["q"], s["q_weight"]), 0.0))
    slot = s["cache_lens"].long()[:, None] + torch.arange(N, device="cuda")
    page, off = s["page_table"].gather(1, slot // c["page"]).long(), slot % c["page"]
    new = {"k_cache": turn(s["k"], s["k_weight"]).to(s["k"].dtype), "v_cache": s["v"]}
    for cache, rows in new.items():  # a node past the request's last writes back what is there
        s[cache][page, off] = torch.where(real[:, :, None, None], rows, s[cache][page, off])
    return s["out"], s["k_cache"], s["v_cache"], s["status"]


def _plain_keep(s):
    c = s["case"]
    j = torch.arange(c["N"], device="cuda")[None]
    kept = j <= s["accepted_len"][:, None]
    to = s["cache_lens"].long()[:, None] + j
    frm = torch.where(kept, s["cache_lens"].long()[:, None] + s["path_nodes"].long(), to)
    frm, to = ((s["page_table"].gather(1, x // c["page"]).long(), x % c["page"]) for x in (frm, to))
    for cache in (s["k_cache"], s["v_cache"]):
        cache[:, to[0], to[1]] = cache[:, frm[0], frm[1]]
    s["new_lens"].copy_(s["cache_lens"] + s["accepted_len"] + 1)
    return s["k_cache"], s["v_cache"], s["new_lens"], s["status"]


def _plain_logits(s):
    c = s["case"]
    B, N, V = c["B"], c["N"], c["V"]
    hist, at = s["history"].long(), torch.arange(c["hist"], device="cuda")[None]
    inside, prompt = at < s["seq_lens"][:, None], at < s["prompt_lens"][:, None]
    one = torch.ones(1, device="cuda")
    said = torch.zeros(B, V + 1, device="cuda").scatter_add_(
        1, torch.where(inside & ~prompt, hist, V), one.expand(B, c["hist"]))
    asked = torch.zeros(B, V + 1, device="cuda").scatter_add_(
        1, torch.where(prompt, hist, V), one.expand(B, c["hist"]))
    path = _ancestors(s)
    path[:, :, 0] = False  # the root is the last verified token: the history has it
    count = said[:, None].repeat(1, N, 1).scatter_add_(
        2, torch.where(path, s["tokens"].long()[:, None], V), one.expand(B, N, N))[..., :V]
    z = s["logits"].float()
    rho, freq, pres = (s[k][:, None, None] for k in ("repetition", "frequency", "presence"))
    seen = (count > 0) | (asked[:, None, :V] > 0)
    z = torch.where(seen, torch.where(z > 0, z / rho, z * rho), z)
    z = z - freq * count - pres * (count > 0)
    if s["bias_tokens"] is not None:
        bias = torch.zeros(B, V, device="cuda").scatter_add_(1, s["bias_tokens"].long(), s["bias_values"])
        z = z + bias[:, None]
    if s["allowed"] is not None:
        bit = torch.arange(32, device="cuda", dtype=torch.int32)
        allowed = ((s["allowed"][..., None] >> bit) & 1).flatten(-2)[..., :V]
        z = torch.where(allowed > 0, z, float("-inf"))
    real = torch.arange(N, device="cuda")[None] < s["n_nodes"][:, None]
    s["out"].copy_(torch.where(real[:, :, None], z, 0.0))
    return s["out"], s["status"]


def _library(s):
    import speculative_decoding_verify_sample_gb300 as sv

    op = s["case"]["op"]
    if op == "attn":
        if "workspace" not in s:
            c = s["case"]
            s["workspace"] = sv.AttentionWorkspace(c["B"], c["N"], c["Hq"], c["Hkv"], c["D"], device="cuda")
        return sv.tree_attention(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["cache_lens"],
                                 s["parents"], s["n_nodes"], out=s["out"], status=s["status"],
                                 workspace=s["workspace"])
    if op == "append":
        q, status = sv.append_nodes(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["page_table"],
                                    s["cache_lens"], s["inv_freq"], s["parents"], s["n_nodes"],
                                    q_weight=s["q_weight"], k_weight=s["k_weight"], eps=1e-6,
                                    interleaved=s["case"]["interleaved"], q_out=s["out"],
                                    status=s["status"])
        return q, s["k_cache"], s["v_cache"], status
    if op == "keep":
        new_lens, status = sv.keep_path(s["path_nodes"], s["accepted_len"], s["k_cache"], s["v_cache"],
                                        s["page_table"], s["cache_lens"], new_lens=s["new_lens"],
                                        status=s["status"])
        return s["k_cache"], s["v_cache"], new_lens, status
    return sv.process_logits(s["logits"], s["history"], s["seq_lens"], s["prompt_lens"],
                             tokens=s["drafts"] if s["case"]["chain"] else s["tokens"],
                             parents=s["parents"], n_nodes=s["n_nodes"],
                             repetition=s["repetition"], frequency=s["frequency"],
                             presence=s["presence"], bias_tokens=s["bias_tokens"],
                             bias_values=s["bias_values"], allowed=s["allowed"], out=s["out"],
                             status=s["status"])


PLAIN = {"attn": _plain_attn, "append": _plain_append, "keep": _plain_keep, "logits": _plain_logits}


def run(state):
    if own:
        return _library(state)
    return PLAIN[state["case"]["op"]](state)


def work(case):
    c = case
    size = 4 if c["dtype"] == "f32" else 2
    lens, nodes = _spread(c["lo"], c["hi"], c["B"]), _spread(c["nlo"], c["N"], c["B"])
    rows = int(nodes.sum())
    if c["op"] == "attn":
        # keys and values once, queries in, rows out; two products for each row and key (which length
        # meets which node count is the seed's: their means stand for it)
        keys = int(lens.sum()) + rows
        return {"bytes": 2 * keys * c["Hkv"] * c["D"] * size + 2 * rows * c["Hq"] * c["D"] * size,
                "flops": 4 * c["Hq"] * c["D"] * float(rows) * (float(lens.mean()) + 1)}
    if c["op"] == "append":
        return {"bytes": 2 * rows * (c["Hq"] + 2 * c["Hkv"]) * c["D"] * size, "flops": 0}
    if c["op"] == "keep":
        # half of the deepest path on average: each kept row in and out, keys and values
        moved = sum(min(c["deep"] / 2, (int(n) - 1) // 2) for n in nodes)
        return {"bytes": int(4 * moved * c["layers"] * c["Hkv"] * c["D"] * size) + 4 * c["B"] * (c["N"] + 4),
                "flops": 0}
    words = rows * (-(-c["V"] // 32)) * 4 if c["mask"] else 0
    return {"bytes": 2 * rows * c["V"] * size + words + 4 * int(lens.sum()), "flops": 0}


def exact(case, seed):
    """The operators from their definitions in 64 bits, request by request."""
    s = prepare(case, seed)
    return {"attn": _exact_attn, "append": _exact_append, "keep": _exact_keep,
            "logits": _exact_logits}[case["op"]](s)


def _chains(s, b):
    """For request b, each node's path from the root to itself, as lists."""
    n = int(s["n_nodes"][b])
    up = [i - 1 for i in range(n)] if s["parents"] is None else s["parents"][b].tolist()[:n]
    paths = []
    for i in range(n):
        paths.append((paths[up[i]] if i else []) + [i])
    return paths


def _slots(s, b, first, last):
    page = s["case"]["page"]
    at = torch.arange(first, last, device="cuda")
    return s["page_table"][b].long()[at // page], at % page


def _exact_attn(s):
    c = s["case"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    G = c["Hq"] // c["Hkv"]
    for b in range(c["B"]):
        paths, first = _chains(s, b), int(s["cache_lens"][b])
        n = len(paths)
        page, off = _slots(s, b, 0, first + n)
        k, v = s["k_cache"][page, off].double(), s["v_cache"][page, off].double()
        hidden = torch.ones(n, first + n, dtype=torch.bool)
        hidden[:, :first] = False
        for i, path in enumerate(paths):
            hidden[i, [first + j for j in path]] = False
        hidden = hidden.cuda()
        for h in range(c["Hq"]):
            x = s["q"][b, :n, h].double() @ k[:, h // G].T / float(c["D"]) ** 0.5
            x[hidden] = float("-inf")
            w = (x - x.max(1, keepdim=True).values).exp()
            out[b, :n, h] = (w @ v[:, h // G]) / w.sum(1, keepdim=True)
    return out, None


def _exact_append(s):
    c = s["case"]
    q_out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    k_out = s["k_cache"].double()
    for b in range(c["B"]):
        paths, first = _chains(s, b), int(s["cache_lens"][b])
        n = len(paths)
        pos = torch.tensor([first + len(p) - 1 for p in paths], dtype=torch.float64, device="cuda")
        page, off = _slots(s, b, first, first + n)
        for name, weight in (("q", s["q_weight"]), ("k", s["k_weight"])):
            x = s[name][b, :n].double().clone()
            if weight is not None:
                x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / c["D"] + 1e-6) * weight.double()
            if s["inv_freq"] is not None:
                half = s["inv_freq"].numel()
                turned = torch.polar(torch.ones_like(pos)[:, None], pos[:, None] * s["inv_freq"].double()[None])
                first_of = [2 * i for i in range(half)] if c["interleaved"] else list(range(half))
                second_of = [2 * i + 1 for i in range(half)] if c["interleaved"] else list(range(half, 2 * half))
                y = torch.complex(x[..., first_of], x[..., second_of]) * turned[:, None]
                x[..., first_of], x[..., second_of] = y.real, y.imag
            if name == "q":
                q_out[b, :n] = x
            else:
                k_out[page, off] = x
    return q_out, k_out, None, None


def _exact_keep(s):
    moved = []
    for cache in (s["k_cache"].double(), s["v_cache"].double()):
        for b in range(s["case"]["B"]):
            first, A = int(s["cache_lens"][b]), int(s["accepted_len"][b])
            page, off = _slots(s, b, first, first + s["case"]["N"])
            path = s["path_nodes"][b, 1:A + 1].long()
            cache[:, page[1:A + 1], off[1:A + 1]] = cache[:, page[path], off[path]]
        moved.append(cache)
    return moved[0], moved[1], None, None


def _exact_logits(s):
    c = s["case"]
    out = torch.zeros(s["logits"].shape, dtype=torch.float64, device="cuda")
    for b in range(c["B"]):
        paths = _chains(s, b)
        total, asked = int(s["seq_lens"][b]), int(s["prompt_lens"][b])
        hist = s["history"][b].long()
        said = torch.bincount(hist[asked:total], minlength=c["V"]).double()
        prompt = torch.bincount(hist[:asked], minlength=c["V"]) > 0
        rho, freq, pres = (float(s[k][b]) for k in ("repetition", "frequency", "presence"))
        for i, path in enumerate(paths):
            count = said + torch.bincount(s["tokens"][b].long()[path[1:]], minlength=c["V"])
            z = s["logits"][b, i].double()
            z = torch.where(prompt | (count > 0), torch.where(z < 0, z * rho, z / rho), z)
            z = z - freq * count - pres * (count != 0).double()
            if s["bias_tokens"] is not None:
                z[s["bias_tokens"][b].long()] += s["bias_values"][b].double()
            if s["allowed"] is not None:
                words = s["allowed"][b, i].cpu().numpy().view(np.uint8)
                bits = np.unpackbits(words, bitorder="little")[:c["V"]].astype(bool)
                z[~torch.from_numpy(bits).cuda()] = float("-inf")
            out[b, i] = z
    return out, None
