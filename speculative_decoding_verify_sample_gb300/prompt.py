"""Binding of the prompt's pass over the paged cache: the norm-rotate-append of a
ragged batch of new tokens, and their attention over the cache.  What these calls
leave there is what the operators on a drafted tree (tree.py) go on from
("Accelerating Sonar through speculation", section "Inferencia con decodificación
especulativa": the target's prefill comes before the first draft).

Shapes, types and devices are checked in csrc/binding.cpp, limits and alignments in
the library; every step runs in its kernels.
"""

from __future__ import annotations

from . import tree
from ._native import lib


def append_chunk(q, k, v, k_cache, v_cache, page_table, cache_lens, cu_tokens, inv_freq=None, *,
                 positions=None, axis_of=None, q_weight=None, k_weight=None, eps=1e-6,
                 interleaved=False, rope_scale=1.0, q_out=None, status=None, stream=None):
    """Norms, rotates and appends the projections of a ragged batch of new tokens.

    q [T, q_heads, D], k and v [T, heads, D] bf16 or f16 (views of one projection
    will do): rows cu_tokens[b] .. cu_tokens[b + 1] - 1 are request b's new
    tokens (``cu_tokens`` [B + 1] int32; none is fine), and its i-th goes to cache
    slot cache_lens[b] + i.  k_cache, v_cache, page_table, cache_lens, weights,
    ``eps``, ``interleaved`` and ``rope_scale`` as in append_nodes.  Pair j of a
    head turns by positions[axis_of[j], t] * inv_freq[j]: ``positions`` [axes, T]
    (or [T]) int32 of any sign, ``axis_of`` [len(inv_freq)] int32 the axis of each
    pair (time, height, width; None: axis 0 of one).  Without positions a
    request's slots are its positions.  Returns (q_out, status [B] int32: 0 or
    DEV_* bits); rows of no request are left as they were (zeros in a new
    q_out).  ``q_out`` may be q.  Asynchronous."""
    return tree._call("spec_append_chunk", (tree._binding or tree.load()).append_chunk, k_cache,
                      stream, q, k, v, k_cache, v_cache, page_table, cache_lens, cu_tokens, inv_freq,
                      positions, axis_of, q_weight, k_weight, eps, interleaved, rope_scale, q_out,
                      status)


class ChunkWorkspace:
    """Device workspace for chunk_attention over requests of up to ``longest`` new
    tokens.  Calls that may run at the same time (on two streams, or two captured
    graphs that may be replayed together) need one each."""

    def __init__(self, longest: int, q_heads: int, kv_heads: int, head_dim: int, device=None):
        import torch
        self.nbytes = int(lib().specv_chunk_workspace_bytes(longest, q_heads, kv_heads, head_dim))
        if self.nbytes == 0:
            raise ValueError(f"unsupported chunk shape longest={longest} q_heads={q_heads} "
                             f"kv_heads={kv_heads} head_dim={head_dim}")
        self.tensor = torch.empty(self.nbytes, dtype=torch.uint8, device=device)


def chunk_attention(q, k_cache, v_cache, page_table, cache_lens, cu_tokens, *, longest=None,
                    scale=None, cap=None, window=None, prefix_lens=None, slopes=None, out=None,
                    status=None, workspace=None, stream=None):
    """Attention of a ragged batch of new tokens over a paged cache.

    q [T, q_heads, D] bf16 or f16, packed by ``cu_tokens`` [B + 1] int32 as in
    append_chunk, whose keys and values are in slots cache_lens[b] + i of
    k_cache, v_cache [pages, page_size, heads, D] already; q_heads a multiple of
    heads.  The token at position p = cache_lens[b] + i sees its request's slots
    s <= p, with ``window`` only those with p - s < window, and with
    ``prefix_lens`` [B] int32 all s < prefix_lens[b] besides (a prompt that sees
    itself whole, or first tokens that a window keeps).  Scores are multiplied by
    ``scale`` (1/sqrt(D)), then capped to cap * tanh(score / cap), then lose
    slopes[h] * |p - s| (``slopes`` [q_heads] f32).  ``longest``: no request has
    more new tokens (None: T; the host's own number saves work where most requests
    have few).  Pages of which no token sees a slot need not exist.  Returns (out
    [T, q_heads, D], status [B] int32: 0 or DEV_* bits); rows of no request are
    left as they were (zeros in a new out).  Asynchronous."""
    return tree._call("spec_chunk_attention", (tree._binding or tree.load()).chunk_attention,
                      k_cache, stream, q, k_cache, v_cache, page_table, cache_lens, cu_tokens,
                      longest, scale, cap, window, prefix_lens, slopes, out, status,
                      None if workspace is None else workspace.tensor)
