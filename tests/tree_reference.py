"""Plain 64-bit forms of the operators on a drafted tree, and their inputs."""

import numpy as np
import torch

# half a step of each type, relative to the value
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def random_parents(rng, B, N):
    parents = np.full((B, N), -1, np.int32)
    for i in range(1, N):
        parents[:, i] = rng.integers(0, i, size=B)
    return parents


def path_of(parents, b, i):
    """Nodes from the root to node i; parents None is a chain."""
    if parents is None:
        return list(range(i + 1))
    path = [i]
    while path[-1] != 0:
        path.append(int(parents[b, path[-1]]))
    return path[::-1]


def make_cache(rng_seed, B, N, Hkv, D, page, lens, dtype, device, *, layout="rows", extra=1,
               fill=float("nan")):
    """A paged cache whose unused places hold `fill`, the verified slots normal
    values; returns (k, v, table).  layout: "rows" [pages, page, H, D];
    "heads" stored [pages, H, page, D]; "pairs" k and v of a page together."""
    gen = torch.Generator(device=device).manual_seed(rng_seed)
    P = max(1, -(-(max(lens) + N) // page)) + 1
    pages = B * P + extra
    if layout == "rows":
        k, v = (torch.full((pages, page, Hkv, D), fill, dtype=dtype, device=device) for _ in "kv")
    elif layout == "heads":
        k, v = (torch.full((pages, Hkv, page, D), fill, dtype=dtype, device=device).transpose(1, 2)
                for _ in "kv")
    else:
        both = torch.full((pages, 2, page, Hkv, D), fill, dtype=dtype, device=device)
        k, v = both[:, 0], both[:, 1]
    table = torch.randperm(pages, generator=gen, device=device)[:B * P].view(B, P).to(torch.int32)
    for b, n in enumerate(lens):
        at = torch.arange(n, device=device)
        pg = table[b].long()[at // page]
        for c in (k, v):
            c[pg, at % page] = torch.randn(n, Hkv, D, generator=gen, device=device).to(dtype)
    return k, v, table


def slots(table, b, page, at, device):
    at = torch.as_tensor(at, device=device, dtype=torch.long)
    return table[b].long()[at // page], at % page


def attention(q, k, v, table, lens, parents, nodes, scale):
    """(out, tolerance parts): out [B, N, Hq, D] in 64 bits (NaN behind the
    last node), mass = sum_j p_j |v_j|, reach = the largest sum |q_d k_d| scale,
    spread = sum_j |v_j| / sum of exp(s_j - max)."""
    B, N, Hq, D = q.shape
    page, Hkv = k.shape[1], k.shape[2]
    out = torch.full(q.shape, float("nan"), dtype=torch.float64, device=q.device)
    mass, reach, spread = out.clone(), out.clone(), out.clone()
    for b in range(B):
        for i in range(int(nodes[b])):
            seen = list(range(int(lens[b]))) + [int(lens[b]) + j for j in path_of(parents, b, i)]
            pg, off = slots(table, b, page, seen, q.device)
            kk = k[pg, off].double().repeat_interleave(Hq // Hkv, 1)
            vv = v[pg, off].double().repeat_interleave(Hq // Hkv, 1)
            qq = q[b, i].double()
            s = torch.einsum("hd,jhd->hj", qq, kk) * scale
            p = torch.softmax(s, -1)
            out[b, i] = torch.einsum("hj,jhd->hd", p, vv)
            mass[b, i] = torch.einsum("hj,jhd->hd", p, vv.abs())
            reach[b, i] = (torch.einsum("hd,jhd->hj", qq.abs(), kk.abs()) * scale).amax(-1)[:, None]
            total = torch.exp(s - s.amax(-1, keepdim=True)).sum(-1)
            spread[b, i] = vv.abs().sum(0) / total[:, None]
    return out, mass, reach, spread


def attention_of_many(q, k, v, table, lens, parents, nodes, scale):
    """attention() for finite caches of many keys: a request at a time."""
    B, N, Hq, D = q.shape
    page, G = k.shape[1], Hq // k.shape[2]
    out = torch.full(q.shape, float("nan"), dtype=torch.float64, device=q.device)
    mass, reach, spread = out.clone(), out.clone(), out.clone()
    for b in range(B):
        n, first = int(nodes[b]), int(lens[b])
        seen = torch.zeros(n, first + n, dtype=torch.bool)
        seen[:, :first] = True
        for i in range(n):
            seen[i, [first + j for j in path_of(parents, b, i)]] = True
        seen = seen.to(q.device)
        pg, off = slots(table, b, page, list(range(first + n)), q.device)
        kk, vv = k[pg, off].double(), v[pg, off].double()
        for h in range(Hq):
            qq, kh, vh = q[b, :n, h].double(), kk[:, h // G], vv[:, h // G]
            s = (qq @ kh.T * scale).masked_fill(~seen, float("-inf"))
            p = torch.softmax(s, -1)
            total = torch.exp(s - s.amax(-1, keepdim=True)).sum(-1, keepdim=True)
            out[b, :n, h], mass[b, :n, h] = p @ vh, p @ vh.abs()
            far = (qq.abs() @ kh.abs().T * scale).masked_fill(~seen, 0.0)
            reach[b, :n, h] = far.amax(-1, keepdim=True)
            spread[b, :n, h] = seen.double() @ vh.abs() / total
    return out, mass, reach, spread


def attention_tolerance(parts, D, keys, dtype):
    """Bound on |kernel - out|, element by element.

    Weights rounded to the cache's type: half a step of each, so at most
    half_step * mass (in f16 also 2^-25, half its smallest step, per weight of
    a row whose largest is at least 1).  Scores: D products and sums in 32
    bits, the matrix unit's sums cut off instead of rounded (2^-23 a sum), and
    the exponent's own rounding: an absolute error e moves a weight by the
    factor 1 +- e, and the sum of weights as much.  Sums over the keys:
    2^-23 a sum over at most keys terms of each 128-key tile and tiles.  The
    result is rounded once."""
    out, mass, reach, spread = parts
    half = HALF_STEP[dtype]
    score = reach * (D + 16) * 2.0 ** -23
    sums = (256 + keys / 64) * 2.0 ** -23
    tol = mass * (half + 2 * score + sums) + half * out.abs() * 1.01 + 2.0 ** -25
    if dtype == torch.float16:
        tol = tol + spread * 2.0 ** -25
    return tol


def append(x, pos, weight, eps, inv_freq, interleaved, rope_scale):
    """x [..., H, D] at positions pos [...], in 64 bits, with the size of the
    terms that each element adds up."""
    x = x.double().clone()
    D = x.shape[-1]
    if weight is not None:
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / D + eps) * weight.double()
    size = x.abs()
    if inv_freq is not None:
        half = inv_freq.numel()
        a = list(range(0, 2 * half, 2)) if interleaved else list(range(half))
        c = list(range(1, 2 * half, 2)) if interleaved else list(range(half, 2 * half))
        t = pos[..., None, None].double() * inv_freq.double()
        xa, xc = x[..., a], x[..., c]
        size[..., a] = size[..., c] = (xa.abs() + xc.abs()) * abs(rope_scale)
        x[..., a] = (xa * t.cos() - xc * t.sin()) * rope_scale
        x[..., c] = (xc * t.cos() + xa * t.sin()) * rope_scale
    return x, size


def append_tolerance(ref, size, dtype):
    """Rounded once to the type; before that the norm (a sum of up to 128
    squares, a root, two products), an angle known to 2^-22 of a turn's
    radius, and two products and a sum, all in 32 bits: 2^-17 of the terms'
    size holds 128 steps of 2^-24."""
    return HALF_STEP[dtype] * ref.abs() * 1.01 + size * 2.0 ** -17 + 2.0 ** -25


def logits(z, history, seq_lens, prompt_lens, tokens, parents, nodes, rho, freq, pres, bias_tokens,
           bias_values, allowed):
    """numpy, row by row: (out in 64 bits, size of the terms); rows behind the
    last stay NaN.  tokens: tree form [B, R] or a chain's [B, R - 1]."""
    B, R, V = z.shape
    out = np.full(z.shape, np.nan)
    size = np.zeros(z.shape)
    for b in range(B):
        total, prompt = int(seq_lens[b]), int(prompt_lens[b]) if prompt_lens is not None else 0
        for i in range(int(nodes[b])):
            path = path_of(parents, b, i)[1:]
            drafted = [int(tokens[b, j] if parents is not None else tokens[b, j - 1]) for j in path]
            said = np.bincount(np.concatenate([history[b, prompt:total], drafted]).astype(np.int64),
                               minlength=V).astype(np.float64)
            text = (said > 0) | (np.bincount(history[b, :prompt], minlength=V) > 0)
            x = z[b, i].astype(np.float64)
            r = float(rho[b]) if rho is not None else 1.0
            f = float(freq[b]) if freq is not None else 0.0
            p = float(pres[b]) if pres is not None else 0.0
            with np.errstate(invalid="ignore"):
                x = np.where(text, np.where(x > 0, x / r, x * r), x)
                size[b, i] = np.abs(x) + abs(f) * said + abs(p)
                x = x - np.where(said > 0, f * said + p, 0.0)
                if bias_tokens is not None:
                    for t, w in zip(bias_tokens[b], bias_values[b]):
                        if t >= 0:
                            x[t] += float(w)
                            size[b, i, t] += abs(float(w))
            if allowed is not None:
                bits = np.unpackbits(np.ascontiguousarray(allowed[b, i]).view(np.uint8),
                                     bitorder="little")[:V].astype(bool)
                x = np.where(bits, x, -np.inf)
            out[b, i] = x
    return out, size


def logits_tolerance(ref, size, dtype):
    """Five operations in 32 bits on terms of `size` (a bias listed up to three
    times: three more), then one rounding to the type."""
    half = 0.0 if dtype == torch.float32 else HALF_STEP[dtype]
    return np.where(np.isfinite(ref), np.abs(np.where(np.isfinite(ref), ref, 0.0)) * half * 1.01, 0.0) \
        + np.where(np.isfinite(size), size, 0.0) * 8 * 2.0 ** -24 + 1e-38
