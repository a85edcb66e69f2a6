"""Timed cases of the operators before the verification: the prompt's pass over
the paged cache, and the drafting of a tree level by level.

Four operators, each in its plain form (elementary torch operations in 32 or 64
bits, rounded once at the end) and through the library's entry points:

  append_chunk     norms of queries and keys per head, the rotation by one or
                   several axes' positions, and the write of a ragged batch of
                   new tokens into the cache
  chunk_attention  attention of those tokens over the cache: causal, with a
                   window, a prefix that all see, capped scores, a bias that
                   falls with the distance
  select_beams     the best of all beams' next tokens by their summed log
                   probabilities: a level of a drafted tree, a beam search's step
  reorder_beams    every beam's states moved to the beams that go on from it

`own` selects the side: False runs the plain forms, True the library.
"""

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    attn = dict(op="attn", page=64, cap=0.0, window=0, prefix=0, slopes=False)
    return [
        # one user, the next token of a conversation, capped scores: latency
        dict(attn, name="attn-one-token", dtype="bf16", B=1, nlo=1, nhi=1, lo=4001, hi=4001, Hq=32, Hkv=8,
             D=128, page=16, cap=50.0),
        # six new prompts, nothing in the cache yet
        dict(attn, name="attn-first-chunk", dtype="bf16", B=6, nlo=517, nhi=4093, lo=0, hi=0, Hq=32, Hkv=8,
             D=128),
        # a served batch: single tokens beside chunks, a window with its first tokens kept
        dict(attn, name="attn-mixed-batch", dtype="f16", B=48, nlo=1, nhi=257, lo=33, hi=8111, Hq=32, Hkv=8,
             D=128, page=32, window=1024, prefix=4),
        # one user's long document, its last chunk
        dict(attn, name="attn-long-document", dtype="bf16", B=1, nlo=4093, nhi=4093, lo=28673, hi=28673,
             Hq=32, Hkv=8, D=128),
        # capped scores under a window, few query heads to a key head
        dict(attn, name="attn-capped-window", dtype="bf16", B=4, nlo=1501, nhi=2049, lo=1023, hi=6143, Hq=16,
             Hkv=8, D=128, cap=50.0, window=4096),
        # a bias by distance, a key head to every query head, narrow heads
        dict(attn, name="attn-distance-bias", dtype="bf16", B=8, nlo=300, nhi=1537, lo=0, hi=2049, Hq=16,
             Hkv=16, D=64, slopes=True),
        # one prompt's projections, text alone: one axis, norms
        dict(name="append-prompt", op="append", dtype="bf16", B=1, nlo=517, nhi=517, lo=0, hi=0, Hq=32, Hkv=8,
             D=128, page=16, axes=1, rot=128, interleaved=False, norm=True),
        # a batch of videos: time, height and width
        dict(name="append-video-batch", op="append", dtype="bf16", B=16, nlo=513, nhi=4093, lo=0, hi=60013,
             Hq=32, Hkv=8, D=128, page=64, axes=3, rot=128, interleaved=False, norm=True),
        # one user's tree grows by a level of eight nodes
        dict(name="select-one-tree", op="select", dtype="bf16", B=1, W=8, K=8, V=128256, ended=False),
        # a served batch of beam searches, some beams ended
        dict(name="select-batch", op="select", dtype="f32", B=64, W=8, K=8, V=128256, ended=True),
        # one user's beams: features of three layers and the text
        dict(name="reorder-one-tree", op="reorder", dtype="bf16", B=1, W=8, K=8, H=12288, L=2048, P=128),
        # a served batch of them
        dict(name="reorder-batch", op="reorder", dtype="bf16", B=64, W=8, K=8, H=12288, L=8192, P=512),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "append", "select", "reorder"])
    dtype = rng.choice(["bf16", "f16"])
    page = rng.choice([1, 8, 16, 24, 32, 64, 100, 128])
    if op in ("attn", "append"):
        B, Hkv, D = _log(rng, 1, 48), rng.choice([1, 2, 4, 8]), rng.choice([64, 64, 80, 96, 128, 128, 128])
        nhi = _log(rng, 1, 4093)
        c = dict(op=op, dtype=dtype, B=B, nlo=rng.choice([nhi, 1 + nhi // 2, 1 + nhi // 50]), Hkv=Hkv, D=D,
                 page=page)
        if op == "attn":
            Hq = Hkv * rng.choice([1, 2, 3, 4, 5, 7, 8])
            nhi = min(nhi, max(1, 6 * 4093 // B))
            # the padded scores of the plain form bound the keys
            hi = min(_log(rng, 1, 28673), max(1, 32 * 4093 * 28673 // (B * Hq * nhi) - nhi))
            window = rng.choice([0, 0, _log(rng, 1, 4096)])
            return dict(c, nlo=min(c["nlo"], nhi), nhi=nhi, lo=rng.choice([0, hi // 2, hi]), hi=hi, Hq=Hq,
                        cap=rng.choice([0.0, 0.0, 20.0, 50.0]), window=window,
                        prefix=rng.choice([0, 4, _log(rng, 1, 600)]), slopes=rng.random() < 0.3)
        nhi = min(nhi, 16 * 2300 // B)
        hi = _log(rng, 1, 60013)
        axes, rot = rng.choice([1, 2, 3, 3]), rng.choice([D, D, D // 2, 0])
        return dict(c, nlo=min(c["nlo"], nhi), nhi=nhi, lo=rng.choice([0, hi // 3]), hi=hi,
                    Hq=Hkv * rng.choice([1, 2, 4, 5]), axes=axes if rot else 1, rot=rot,
                    interleaved=rng.random() < 0.5, norm=rng.random() < 0.6)
    W = rng.randint(1, 16)
    K = rng.choice([W, W, rng.randint(1, 32)])
    B = _log(rng, 1, max(1, 512 // W))
    if op == "select":
        return dict(op=op, dtype=rng.choice(["bf16", "f32"]), B=B, W=W, K=K,
                    V=rng.choice([1024, 32003, 50000, 128256]), ended=rng.random() < 0.5)
    return dict(op=op, dtype=dtype, B=B, W=W, K=K, H=8 * _log(rng, 1, 1536), L=_log(rng, 1, 8192),
                P=_log(rng, 1, 512))


def _spread(lo, hi, B):
    """B whole numbers from lo to hi, evenly."""
    return np.rint(np.linspace(lo, hi, B)).astype(np.int64) if B > 1 else np.array([hi])


def _lengths(c):
    """New tokens and cached tokens of each request: the case's own, whatever the seed."""
    rs = np.random.RandomState(7)
    return rs.permutation(_spread(c["nlo"], c["nhi"], c["B"])), rs.permutation(_spread(c["lo"], c["hi"], c["B"]))


def _put(a, dtype=None):
    return torch.from_numpy(np.ascontiguousarray(a, dtype)).cuda()


def prepare(case, seed):
    c, rs = dict(case), np.random.RandomState(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt, B = DTYPES[c["dtype"]], c["B"]
    s = dict(case=c, status=torch.zeros(B, dtype=torch.int32, device="cuda"))

    def normal(*shape, scale=1.0, dtype=dt):
        return torch.randn(*shape, generator=gen, device="cuda").mul_(scale).to(dtype)

    if c["op"] in ("attn", "append"):
        new, lens = _lengths(c)
        order = rs.permutation(B)  # the seed says which request is which
        new, lens = new[order], lens[order]
        T, Hq, Hkv, D, page = int(new.sum()), c["Hq"], c["Hkv"], c["D"], c["page"]
        cu = np.concatenate([[0], np.cumsum(new)])
        first = lens // page if c["op"] == "append" else lens * 0  # append: the chunk's own pages alone
        used = (lens + new - 1) // page - first + 1
        P = int((first + used).max())
        table = np.zeros((B, P), np.int64)
        ids, at = rs.permutation(int(used.sum())), np.cumsum(used) - used
        for b in range(B):
            table[b, first[b]:first[b] + used[b]] = ids[at[b]:at[b] + used[b]]
        s.update(page_table=_put(table, np.int32), cache_lens=_put(lens, np.int32), cu_tokens=_put(cu, np.int32),
                 longest=int(new.max()), slots=int((lens + new).max()))
        for name in ("k_cache", "v_cache"):
            s[name] = normal(int(used.sum()), page, Hkv, D)
        # the projection's output, queries, keys and values side by side in one row
        qkv = normal(T, (Hq + 2 * Hkv) * D)
        q, k, v = qkv.split([Hq * D, Hkv * D, Hkv * D], dim=-1)
        s.update(q=q.unflatten(-1, (Hq, D)), k=k.unflatten(-1, (Hkv, D)), v=v.unflatten(-1, (Hkv, D)),
                 out=torch.zeros(T, Hq, D, dtype=dt, device="cuda"))
    if c["op"] == "attn":
        s["slopes"] = _put(2.0 ** (-8.0 * np.arange(1, Hq + 1) / Hq), np.float32) if c["slopes"] else None
        s["prefix_lens"] = None
        if c["prefix"]:  # never behind a request's last slot
            s["prefix_lens"] = _put(np.minimum(c["prefix"], lens + new), np.int32)
    if c["op"] == "append":
        half = c["rot"] // 2
        s["inv_freq"] = _put(500000.0 ** (-np.arange(half) / max(half, 1)), np.float32) if half else None
        s["q_weight"] = (1 + normal(D, scale=0.1, dtype=torch.float32)).to(dt) if c["norm"] else None
        s["k_weight"] = (1 + normal(D, scale=0.1, dtype=torch.float32)).to(dt) if c["norm"] else None
        s["positions"] = s["axis_of"] = None
        if c["axes"] > 1:
            # text, then frames of patches: the time goes on, height and width begin again in each
            i = np.arange(T) - np.repeat(cu[:-1], new) + np.repeat(lens, new)
            side = int(rs.randint(14, 25))
            grid = np.stack([i // side ** 2, i // side % side, i % side])[-c["axes"]:]
            s["positions"] = _put(grid, np.int32)
            # pairs shared out in runs, the first axis a little shorter
            cuts = np.cumsum([half // 4] + [(half - half // 4) // (c["axes"] - 1)] * (c["axes"] - 1))
            s["axis_of"] = _put(np.minimum(np.searchsorted(cuts, np.arange(half), side="right"), c["axes"] - 1),
                                np.int32)
    if c["op"] == "select":
        W, K, V = c["W"], c["K"], c["V"]
        s["logits"] = normal(B, W, V, scale=3.0)
        s["scores"] = _put(-rs.exponential(4.0, (B, W)), np.float32)
        s["ended"] = _put(rs.random_sample((B, W)) < 0.2, np.int32) if c["ended"] else None
        s.update(out_scores=torch.zeros(B, K, device="cuda"),
                 tokens=torch.zeros(B, K, dtype=torch.int32, device="cuda"),
                 beams=torch.zeros(B, K, dtype=torch.int32, device="cuda"))
    if c["op"] == "reorder":
        W, K = c["W"], c["K"]
        # a few beams have most of the children, as the best scores do; some places stay empty
        pick = np.minimum(rs.exponential(0.35 * W, (B, K)).astype(np.int64), W - 1)
        s["beams"] = _put(np.where(rs.random_sample((B, K)) < 0.05, -1, pick), np.int32)
        s["states"] = [normal(B, W, c["H"]),
                       torch.randint(0, 128256, (B, W, c["L"]), generator=gen, device="cuda", dtype=torch.int32),
                       torch.randint(0, 65536, (B, W, c["P"]), generator=gen, device="cuda", dtype=torch.int32)]
        s["out"] = [torch.zeros(B, K, x.shape[2], dtype=x.dtype, device="cuda") for x in s["states"]]
    return s


def _places(s):
    """[B, N]: the packed row of each request's i-th new token, and whether there is one."""
    cu = s["cu_tokens"].long()
    i = torch.arange(s["longest"], device="cuda")
    row = cu[:-1, None] + i
    return row.clamp(max=int(s["q"].shape[0]) - 1), row < cu[1:, None]


def _plain_attn(s):
    c = s["case"]
    B, Hq, Hkv, D = (c[k] for k in ("B", "Hq", "Hkv", "D"))
    G, N, L = Hq // Hkv, s["longest"], s["slots"]
    row, real = _places(s)
    slot = torch.arange(L, device="cuda")
    page, off = s["page_table"].long()[:, slot // c["page"]], slot % c["page"]  # a page behind the last is page 0
    k = s["k_cache"][page, off].float()
    q = s["q"][row].float().reshape(B, N, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, N * G, D)
    scores = (q @ k.permute(0, 2, 3, 1)).mul_(D ** -0.5)
    del k
    if c["cap"]:
        scores.div_(c["cap"]).tanh_().mul_(c["cap"])
    pos = s["cache_lens"].long()[:, None] + torch.arange(N, device="cuda")
    back = pos[:, :, None] - slot  # how far behind the token the slot is
    view = scores.view(B, Hkv, N, G, L)
    if s["slopes"] is not None:
        view.addcmul_(back.abs().float()[:, None, :, None], s["slopes"].view(1, Hkv, 1, G, 1), value=-1.0)
    seen = back >= 0
    if c["window"]:
        seen &= back < c["window"]
    if s["prefix_lens"] is not None:
        seen |= slot < s["prefix_lens"].long()[:, None, None]
    seen |= ~real[:, :, None]  # rows that are no token's: left out below
    view.masked_fill_(~seen[:, None, :, None], float("-inf"))
    del seen, back
    scores -= scores.amax(-1, keepdim=True)
    scores.exp_()
    scores /= scores.sum(-1, keepdim=True)
    v = s["v_cache"][page, off].float()
    o = (scores @ v.permute(0, 2, 1, 3)).reshape(B, Hkv, N, G, D).permute(0, 2, 1, 3, 4).reshape(B, N, Hq, D)
    s["out"].copy_(o[real])
    return s["out"], s["status"]


def _plain_append(s):
    c = s["case"]
    D, T = c["D"], s["q"].shape[0]
    row = torch.arange(T, device="cuda")
    b = (row[:, None] >= s["cu_tokens"].long()[1:]).sum(1)
    slot = s["cache_lens"].long()[b] + row - s["cu_tokens"].long()[b]

    def turn(x, weight):
        x = x.float()
        if weight is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * weight.float()
        if s["inv_freq"] is None:
            return x
        half = s["inv_freq"].numel()
        pos = slot[:, None] if s["positions"] is None else s["positions"].long()[s["axis_of"].long()].T
        angle = pos[:, None].double() * s["inv_freq"].double()
        cos, sin = angle.cos().float(), angle.sin().float()
        if c["interleaved"]:
            a, d = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
            both = torch.stack([a * cos - d * sin, d * cos + a * sin], -1).flatten(-2)
        else:
            a, d = x[..., :half], x[..., half:2 * half]
            both = torch.cat([a * cos - d * sin, d * cos + a * sin], -1)
        return torch.cat([both, x[..., 2 * half:]], -1)

    s["out"].copy_(turn(s["q"], s["q_weight"]))
    page, off = s["page_table"].long()[b, slot // c["page"]], slot % c["page"]
    s["k_cache"][page, off] = turn(s["k"], s["k_weight"]).to(s["k"].dtype)
    s["v_cache"][page, off] = s["v"]
    return s["out"], s["k_cache"], s["v_cache"], s["status"]


def _plain_select(s):
    c = s["case"]
    B, W, K, V = (c[k] for k in ("B", "W", "K", "V"))
    # in 64 bits: which of two near scores is larger decides a token
    z = s["logits"].double()
    z -= z.amax(-1, keepdim=True)
    z -= z.exp().sum(-1, keepdim=True).log()
    z += s["scores"].double()[:, :, None]
    if s["ended"] is not None:  # one candidate, with the score that it has: its token is 2
        over = s["ended"] != 0
        z.masked_fill_(over[:, :, None], float("-inf"))
        z[:, :, 2] = torch.where(over, s["scores"].double(), z[:, :, 2])
    best, at = torch.sort(z.flatten(1), dim=1, descending=True, stable=True)
    best, at = best[:, :K], at[:, :K]
    empty = best == float("-inf")
    s["out_scores"].copy_(best)
    s["tokens"].copy_(torch.where(empty, -1, at % V))
    s["beams"].copy_(torch.where(empty, -1, at // V))
    return s["out_scores"], s["tokens"], s["beams"], s["status"]


def _plain_reorder(s):
    B = s["case"]["B"]
    at = torch.arange(B, device="cuda")[:, None]
    there = s["beams"] >= 0

    def moved(x, out):
        out.copy_(torch.where(there[:, :, None], x[at, s["beams"].long().clamp(min=0)], out))
        return out

    return (*map(moved, s["states"], s["out"]), s["status"])


def _library(s):
    import speculative_decoding_verify_sample_gb300 as sv

    c = s["case"]
    if c["op"] == "attn":
        if "workspace" not in s:
            s["workspace"] = sv.ChunkWorkspace(s["longest"], c["Hq"], c["Hkv"], c["D"], device="cuda")
        return sv.chunk_attention(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["cache_lens"],
                                  s["cu_tokens"], longest=s["longest"], cap=c["cap"] or None,
                                  window=c["window"] or None, prefix_lens=s["prefix_lens"],
                                  slopes=s["slopes"], out=s["out"], status=s["status"],
                                  workspace=s["workspace"])
    if c["op"] == "append":
        q, status = sv.append_chunk(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["page_table"],
                                    s["cache_lens"], s["cu_tokens"], s["inv_freq"],
                                    positions=s["positions"], axis_of=s["axis_of"], q_weight=s["q_weight"],
                                    k_weight=s["k_weight"], eps=1e-6, interleaved=c["interleaved"],
                                    q_out=s["out"], status=s["status"])
        return q, s["k_cache"], s["v_cache"], status
    if c["op"] == "select":
        if "workspace" not in s:
            s["workspace"] = sv.BeamWorkspace(c["B"], c["W"], c["K"], c["V"], device="cuda")
        return sv.select_beams(s["logits"], s["scores"], c["K"], ended=s["ended"], end_token=2,
                               out_scores=s["out_scores"], tokens=s["tokens"], beams=s["beams"],
                               status=s["status"], workspace=s["workspace"])
    outs, status = sv.reorder_beams(s["beams"], s["states"], out=s["out"], status=s["status"])
    return (*outs, status)


PLAIN = {"attn": _plain_attn, "append": _plain_append, "select": _plain_select, "reorder": _plain_reorder}


def run(state):
    if own:
        return _library(state)
    return PLAIN[state["case"]["op"]](state)


def work(case):
    c = case
    size = 4 if c["dtype"] == "f32" else 2
    if c["op"] in ("attn", "append"):
        new, lens = _lengths(c)
        T, width = int(new.sum()), c["D"] * size
        if c["op"] == "append":
            return {"bytes": 2 * T * (c["Hq"] + 2 * c["Hkv"]) * width, "flops": 0}
        pairs, rows = 0, 0
        window = c["window"] or 1 << 40
        for n, len_ in zip(new, lens):
            pos = np.arange(len_, len_ + n)
            prefix = min(c["prefix"], int(len_ + n))
            first = np.maximum(0, pos - window + 1)  # of the slots that its window lets a token see
            pairs += int((pos + 1 - first).sum() + np.where(pos < prefix, prefix - 1 - pos, 0).sum()
                         + np.minimum(first, prefix).sum())
            rows += int(len_ + n - first[0]) + min(prefix, int(first[0]))
        return {"bytes": 2 * rows * c["Hkv"] * width + 2 * T * c["Hq"] * width,
                "flops": 4 * c["Hq"] * c["D"] * float(pairs)}
    if c["op"] == "select":  # the rows that go on: all but a fifth of them where some have ended
        rows = c["B"] * c["W"] * (0.8 if c["ended"] else 1.0)
        return {"bytes": rows * c["V"] * size + 4 * c["B"] * (2 * c["W"] + 3 * c["K"]), "flops": 0}
    # written: 95 of 100 places; read: each beam that has a child, once (the chances that prepare() gives)
    W, K = c["W"], c["K"]
    share = np.diff(np.append(1 - np.exp(-np.arange(W) / (0.35 * W)), 1.0))
    used = float((1 - (1 - 0.95 * share) ** K).sum())
    row = c["H"] * size + 4 * (c["L"] + c["P"])
    return {"bytes": c["B"] * (used + 0.95 * K) * row, "flops": 0}


def exact(case, seed):
    """The operators from their definitions in 64 bits, request by request."""
    s = prepare(case, seed)
    return {"attn": _exact_attn, "append": _exact_append, "select": _exact_select,
            "reorder": _exact_reorder}[case["op"]](s)


def _rows_of(s, b):
    """Request b's packed rows, and the pages and rows of its slots up to the last."""
    first, last = s["cu_tokens"][b:b + 2].tolist()
    done = int(s["cache_lens"][b])
    at = torch.arange(done + last - first, device="cuda")
    page = s["case"]["page"]
    return first, last, done, s["page_table"][b].long()[at // page], at % page


def _exact_attn(s):
    c = s["case"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    group = c["Hq"] // c["Hkv"]
    for b in range(c["B"]):
        first, last, done, page, off = _rows_of(s, b)
        k, v = s["k_cache"][page, off].double(), s["v_cache"][page, off].double()
        here = torch.arange(done, done + last - first, device="cuda")[:, None]
        there = torch.arange(k.shape[0], device="cuda")[None]
        hidden = there > here
        if c["window"]:
            hidden |= there <= here - c["window"]
        if s["prefix_lens"] is not None:
            hidden &= there >= int(s["prefix_lens"][b])
        for h in range(c["Hq"]):
            x = s["q"][first:last, h].double() @ k[:, h // group].T / float(c["D"]) ** 0.5
            if c["cap"]:
                x = c["cap"] * torch.tanh(x / c["cap"])
            if s["slopes"] is not None:
                x -= float(s["slopes"][h]) * (here - there).abs().double()
            x[hidden] = float("-inf")
            x = (x - x.max(1, keepdim=True).values).exp()
            out[first:last, h] = (x @ v[:, h // group]) / x.sum(1, keepdim=True)
    return out, None


def _exact_append(s):
    c = s["case"]
    q_out, k_out, v_out = s["q"].double(), s["k_cache"].double(), s["v_cache"].double()
    for b in range(c["B"]):
        first, last, done, page, off = _rows_of(s, b)
        page, off = page[done:], off[done:]
        for name, weight in (("q", s["q_weight"]), ("k", s["k_weight"])):
            x = s[name][first:last].double().clone()
            if weight is not None:
                x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / c["D"] + 1e-6) * weight.double()
            half = c["rot"] // 2
            for j in range(half):
                if s["positions"] is None:
                    pos = torch.arange(done, done + last - first, device="cuda").double()
                else:
                    pos = s["positions"][int(s["axis_of"][j]), first:last].double()
                turned = torch.polar(torch.ones_like(pos), pos * s["inv_freq"][j].double())
                at = (2 * j, 2 * j + 1) if c["interleaved"] else (j, j + half)
                y = torch.complex(x[..., at[0]], x[..., at[1]]) * turned[:, None]
                x[..., at[0]], x[..., at[1]] = y.real, y.imag
            if name == "q":
                q_out[first:last] = x
            else:
                k_out[page, off] = x
        v_out[page, off] = s["v"][first:last].double()
    return q_out, k_out, v_out, None


def _exact_select(s):
    c = s["case"]
    out = torch.empty(c["B"], c["K"], dtype=torch.float64, device="cuda")
    for b in range(c["B"]):
        pool = []
        for w in range(c["W"]):
            so_far = float(s["scores"][b, w])
            if s["ended"] is not None and int(s["ended"][b, w]):
                pool.append(torch.full((1,), so_far, dtype=torch.float64, device="cuda"))
            else:
                z = s["logits"][b, w].double()
                pool.append(so_far + (z - torch.logsumexp(z, 0)).topk(min(c["K"], c["V"])).values)
        pool = torch.cat(pool).sort(descending=True).values[:c["K"]]
        out[b] = float("-inf")
        out[b, :pool.numel()] = pool
    return out, None, None, None


def _exact_reorder(s):
    """A move computes nothing: its 16-bit states, in 64 bits."""
    x, beams = s["states"][0].double(), s["beams"].tolist()
    zero = torch.zeros(x.shape[2], dtype=torch.float64, device="cuda")
    kept = [torch.stack([x[b, w] if w >= 0 else zero for w in row]) for b, row in enumerate(beams)]
    return torch.stack(kept), None, None, None
