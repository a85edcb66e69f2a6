"""Plain 64-bit forms of the operators before the verification, and their inputs."""

import numpy as np
import torch

from tree_reference import HALF_STEP, slots


def seen_by(pos, keys, window, prefix, device):
    """[rows, keys]: which slots below `keys` the tokens at positions pos see."""
    s = torch.arange(keys, device=device)[None]
    p = pos[:, None]
    return (s < prefix) | ((s <= p) & (s > p - (window or 1 << 40)))


def attention(q, k, v, table, lens, cu, scale, cap=None, window=None, prefix=None, slopes=None):
    """(out, tolerance) [T, Hq, D] in 64 bits; NaN in rows of no request.

    The tolerance, element by element.  Weights rounded to the cache's type: half a
    step of each, half * sum p|v| (in f16 also 2^-25, half its smallest step, per
    weight of a row whose largest is at least 1).  A score that is e off moves
    its weight by the factor 1 +- e and the sum of weights as much; e has D
    products and sums in 32 bits, the matrix unit's sums cut off instead of
    rounded (2^-23 a sum); the capped score's exponential, sum, reciprocal and
    product (each within 2^-22 of terms of at most the cap: 2^-20 of it together); the
    bias's three roundings; the roundings of score and maximum in the exponent and
    the exponential's own 2^-22.  Sums over the keys: 2^-23 a sum over at most 256
    terms of each pair of 128-key tiles and the tiles.  The result is rounded once."""
    T, Hq, D = q.shape
    page, G, dev = k.shape[1], Hq // k.shape[2], q.device
    half = HALF_STEP[q.dtype]
    out = torch.full(q.shape, float("nan"), dtype=torch.float64, device=dev)
    tol = out.clone()
    for b, done in enumerate(lens):
        first, last = int(cu[b]), int(cu[b + 1])
        n, keys = last - first, int(done) + last - first
        if n <= 0:
            continue
        pos = torch.arange(int(done), keys, device=dev)
        seen = seen_by(pos, keys, window, 0 if prefix is None else int(prefix[b]), dev)
        some = seen.any(0)
        pg, off = slots(table, b, page, list(range(keys)), dev)
        pg = torch.where(some, pg, 0)  # a page that nobody sees need not exist
        kk, vv = k[pg, off].double(), v[pg, off].double()
        kk, vv = (torch.where(some[:, None, None], x, 0.0) for x in (kk, vv))
        away = (pos[:, None] - torch.arange(keys, device=dev)).abs().double()
        for h in range(Hq):
            qq, kh, vh = q[first:last, h].double(), kk[:, h // G], vv[:, h // G]
            y = qq @ kh.T * scale
            e = (qq.abs() @ kh.abs().T) * scale * (D + 16) * 2.0 ** -23
            if cap is not None:
                y = cap * torch.tanh(y / cap)
                e = e + cap * 2.0 ** -20
            if slopes is not None:
                bias = float(slopes[h]) * away
                y = y - bias
                e = e + bias.abs() * 2.0 ** -22
            y = y.masked_fill(~seen, float("-inf"))
            top = y.amax(-1, keepdim=True)
            p = torch.softmax(y, -1)
            e = torch.where(seen, e + (y.abs() + top.abs()) * 2.0 ** -22 + 2.0 ** -21, 0.0)
            odd = ~torch.isfinite(vh)
            fine = torch.where(odd, 0.0, vh)
            o = p @ fine
            for j in torch.nonzero(odd.any(-1)).flatten().tolist():  # only for rows that see them
                o = o + torch.where(seen[:, j, None] & odd[j], vh[j], 0.0)
            mass = p @ fine.abs()
            pe = torch.where(seen, p * e, 0.0)
            t = mass * (half + (256 + keys / 64) * 2.0 ** -23) + pe @ fine.abs()
            t = t + o.abs() * (pe.sum(-1, keepdim=True) + half * 1.01) + 2.0 ** -25
            if q.dtype == torch.float16:
                total = torch.exp(y - top).sum(-1, keepdim=True)
                t = t + (seen.double() @ fine.abs()) / total * 2.0 ** -25
            out[first:last, h], tol[first:last, h] = o, t
    return out, tol


def select(logits, scores, K, ended=None, end_token=0):
    """numpy, request by request, in 64 bits: (scores, tokens, beams [B, K], rows), rows[b][w] the
    scores of all of that beam's tokens, None of one that has no row."""
    B, W, V = logits.shape
    out = np.full((B, K), -np.inf)
    tokens, beams = np.full((B, K), -1), np.full((B, K), -1)
    rows = [[None] * W for _ in range(B)]
    for b in range(B):
        parts, names = [], []
        for w in range(W):
            if scores[b, w] == -np.inf:
                continue
            if ended is not None and ended[b, w]:
                parts.append(np.array([float(scores[b, w])]))
                names.append(np.array([[w, end_token]]))
                continue
            z = logits[b, w].astype(np.float64)
            m = z.max()
            if m == -np.inf:
                continue
            rows[b][w] = float(scores[b, w]) + (z - m - np.log(np.exp(z - m).sum()))
            parts.append(rows[b][w])
            names.append(np.stack([np.full(V, w), np.arange(V)], 1))
        if not parts:
            continue
        pool, names = np.concatenate(parts), np.concatenate(names)
        order = np.lexsort((names[:, 1], names[:, 0], -pool))[:K]
        best = order[pool[order] > -np.inf]
        out[b, :len(best)] = pool[best]
        beams[b, :len(best)], tokens[b, :len(best)] = names[best, 0], names[best, 1]
    return out, tokens, beams, rows
