"""Binding of the target's pass over a drafted tree: the norm-rotate-append of
the nodes' projections, the attention over a paged cache, the penalties and
masks on the logits, and the move of the accepted path's cache rows
("Decodificación Especulativa y EAGLE", section "Verificación de Atención en
Árvore"; "Accelerating Sonar through speculation", section "EAGLE").

Shapes, types and devices are checked in csrc/binding.cpp (these calls take a few
microseconds on the device, so what the host spends on them counts), the limits
and alignments in the library; every step runs in its kernels.
"""

from __future__ import annotations

import contextlib
import ctypes
import importlib.machinery
import importlib.util
import os

from ._native import SpecVerifyError, lib
from .build import binding_failure, binding_path

_binding = None


def load():
    """The extension, bound to the library.  Raises if it is not built."""
    global _binding
    if _binding is None:
        path, handle = binding_path(), lib()
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is not built: " + (
                binding_failure() or "run speculative_decoding_verify_sample_gb300.build()"))
        loader = importlib.machinery.ExtensionFileLoader("_binding", path)
        module = importlib.util.module_from_spec(
            importlib.util.spec_from_loader("_binding", loader))
        loader.exec_module(module)
        module.bind(*(ctypes.cast(fn, ctypes.c_void_p).value for fn in (
            handle.spec_append_nodes, handle.spec_tree_attention, handle.spec_keep_path,
            handle.spec_process_logits, handle.specv_attention_workspace_bytes,
            handle.spec_append_chunk, handle.spec_chunk_attention,
            handle.specv_chunk_workspace_bytes, handle.spec_select_beams,
            handle.specv_beam_workspace_bytes, handle.spec_reorder_beams)))
        _binding = module
    return _binding


@contextlib.contextmanager
def _there(device, stream):
    import torch
    with torch.cuda.device(device):
        if stream is None:
            yield
        else:
            if not isinstance(stream, torch.cuda.Stream):
                stream = torch.cuda.ExternalStream(getattr(stream, "cuda_stream", stream), device)
            with torch.cuda.stream(stream):
                yield


def _call(name, fn, tensor, stream, *args):
    """fn(*args) on tensor's device and the stream: its outputs are allocated where
    it launches."""
    cuda = getattr(tensor, "is_cuda", False)
    out = fn(*args) if stream is None or not cuda else None
    if out is None:
        with _there(tensor.device, stream):
            out = fn(*args)
        if out is None:  # the stream took the call to its own device
            raise ValueError(f"stream is of another device than the tensors, on {tensor.device}")
    if out.__class__ is int:
        raise SpecVerifyError(name, out)
    return out


def append_nodes(q, k, v, k_cache, v_cache, page_table, cache_lens, inv_freq=None, parents=None,
                 n_nodes=None, *, q_weight=None, k_weight=None, eps=1e-6, interleaved=False,
                 rope_scale=1.0, q_out=None, status=None, stream=None):
    """Norms, rotates and appends the projections of a drafted tree's nodes.

    q [B, N, q_heads, D], k and v [B, N, heads, D] bf16 or f16 (views of one
    projection will do); k_cache, v_cache [pages, page_size, heads, D];
    page_table [B, P] and cache_lens [B] int32.  Each head of q and k is
    divided by the root of its mean square plus ``eps`` and multiplied by
    ``q_weight`` / ``k_weight`` [D] (16-byte aligned; None: no norm), then its first
    2 * len(inv_freq) elements are rotated by (cache_lens[b] + depth of the
    node) * ``inv_freq`` (f32; None: no rotation), in pairs (2j, 2j + 1) if
    ``interleaved`` and (j, j + len(inv_freq)) if not, and scaled by
    ``rope_scale``.  Node i's key and value go to cache slot
    cache_lens[b] + i.  ``parents`` [B, N] int32 (None: a chain), ``n_nodes``
    [B] int32 (None: all N).  Returns (q_out, status [B] int32: 0 or DEV_*
    bits); rows of q_out behind n_nodes[b] are left as they were (zeros in a
    new one).  ``q_out`` may be q.  Asynchronous."""
    return _call("spec_append_nodes", (_binding or load()).append_nodes, k_cache, stream, q, k, v,
                 k_cache, v_cache, page_table, cache_lens, inv_freq, parents, n_nodes, q_weight,
                 k_weight, eps, interleaved, rope_scale, q_out, status)


class AttentionWorkspace:
    """Device workspace for tree_attention over B requests of up to N nodes.  Calls
    that may run at the same time (on two streams, or two captured graphs that
    may be replayed together) need one each."""

    def __init__(self, B: int, N: int, q_heads: int, kv_heads: int, head_dim: int, device=None):
        import torch
        self.nbytes = int(lib().specv_attention_workspace_bytes(B, N, q_heads, kv_heads, head_dim))
        if self.nbytes == 0:
            raise ValueError(f"unsupported attention shape B={B} N={N} q_heads={q_heads} "
                             f"kv_heads={kv_heads} head_dim={head_dim}")
        self.tensor = torch.empty(self.nbytes, dtype=torch.uint8, device=device)


def tree_attention(q, k_cache, v_cache, page_table, cache_lens, parents=None, n_nodes=None, *,
                   scale=None, out=None, status=None, workspace=None, stream=None):
    """Attention of a drafted tree's nodes over a paged cache.

    q [B, N, q_heads, D] bf16 or f16; k_cache, v_cache [pages, page_size,
    heads, D] with the nodes' own keys and values already in slots
    cache_lens[b] + i (append_nodes); page_table [B, P] int32; q_heads a
    multiple of heads.  Node i of request b sees the cache_lens[b] verified
    slots, itself and its ancestors by ``parents`` [B, N] int32 (None: a
    chain; N = 1 is plain decoding).  ``scale`` (1/sqrt(D)) multiplies the
    scores.  Returns (out [B, N, q_heads, D], status [B] int32: 0 or DEV_*
    bits); rows of out behind n_nodes[b] are left as they were (zeros in a new
    one).  Asynchronous."""
    return _call("spec_tree_attention", (_binding or load()).tree_attention, k_cache, stream, q,
                 k_cache, v_cache, page_table, cache_lens, parents, n_nodes, scale, out, status,
                 None if workspace is None else workspace.tensor)


def keep_path(path_nodes, accepted_len, k_cache, v_cache, page_table, cache_lens, *, new_lens=None,
              status=None, stream=None):
    """Keeps the accepted path's rows of the cache: slot cache_lens[b] + j gets
    the row of slot cache_lens[b] + path_nodes[b, j], j = 1 ..
    accepted_len[b] (the outputs of verify_tree_greedy).  k_cache and v_cache
    may be [layers, pages, page_size, heads, D]: every layer in one call.
    Returns (new_lens [B] = cache_lens + accepted_len + 1, status [B]) int32;
    a flagged request keeps its rows and its length.  Asynchronous."""
    return _call("spec_keep_path", (_binding or load()).keep_path, k_cache, stream, path_nodes,
                 accepted_len, k_cache, v_cache, page_table, cache_lens, new_lens, status)


def process_logits(logits, history, seq_lens, prompt_lens=None, *, tokens=None, parents=None,
                   n_nodes=None, repetition=None, frequency=None, presence=None, bias_tokens=None,
                   bias_values=None, allowed=None, out=None, status=None, stream=None):
    """Penalties, biases and grammar masks on the logits of a drafted tree's
    nodes, before the verification (or, with one row, a sampler).

    logits [B, R, V] (or [B, V]) bf16 or f32: row i is what the target says
    after node i, whose text is history[b, :seq_lens[b]] and the tokens on the
    path from the root to it.  ``tokens``: with ``parents`` [B, R] the nodes'
    tokens [B, R] (node 0's is unused), without (a chain) the drafted tokens
    [B, R - 1] of spec_verify_sample; ``n_nodes`` [B]: rows in use.  int32.
    A token of the text is divided (z > 0) or multiplied by ``repetition``;
    c times in the text from ``prompt_lens`` on, it loses frequency * c +
    presence (f32 [B] each).  ``bias_tokens``, ``bias_values`` [B, n] add a
    bias (a token below 0: an empty place).  ``allowed`` [B, R, ceil(V/32)]
    int32: bit t % 32 of word t // 32 set, or z becomes -inf.  Returns (out,
    status [B] int32: 0 or DEV_* bits); rows behind n_nodes[b] are left as
    they were (zeros in a new out).  ``out`` may be logits.  Asynchronous."""
    return _call("spec_process_logits", (_binding or load()).process_logits, logits, stream, logits,
                 history, seq_lens, prompt_lens, tokens, parents, n_nodes, repetition, frequency,
                 presence, bias_tokens, bias_values, allowed, out, status)
