"""Binding of the target's pass over a drafted tree: the norm-rotate-append of
the nodes' projections, the attention over a paged cache, the penalties and
masks on the logits, and the move of the accepted path's cache rows
("Decodificación Especulativa y EAGLE", section "Verificación de Atención en
Árvore"; "Accelerating Sonar through speculation", section "EAGLE").

As in the rest of the binding: shapes, types and devices are checked here,
the limits and alignments in the library; every step runs in its kernels.
"""

from __future__ import annotations

import contextlib
import ctypes
import math

import torch

from ._native import (SPECV_BF16, SPECV_F16, SPECV_F32, CacheArg, RowsArg, check, lib)

_CACHE_DTYPES = {torch.bfloat16: SPECV_BF16, torch.float16: SPECV_F16}
_LOGIT_DTYPES = {torch.bfloat16: SPECV_BF16, torch.float32: SPECV_F32}
_NOTHING = contextlib.nullcontext()


@contextlib.contextmanager
def _other(device, stream):
    with torch.cuda.device(device):
        if stream is None:
            yield
        else:
            if not isinstance(stream, torch.cuda.Stream):
                stream = torch.cuda.ExternalStream(getattr(stream, "cuda_stream", stream), device)
            with torch.cuda.stream(stream):
                yield


def _on(device, stream):
    """The device and stream that the call allocates on and launches on."""
    if device.type != "cuda":
        raise ValueError(f"the operators on a drafted tree take CUDA tensors, got {device}")
    if stream is None and device.index == torch.cuda.current_device():
        return _NOTHING
    return _other(device, stream)


def _current(device):
    return torch.cuda.current_stream(device).cuda_stream


def _need(name, t, shape, dtype, dev):
    """t is a contiguous tensor of this shape, type and device."""
    if not isinstance(t, torch.Tensor) or t.shape != shape or t.dtype != dtype or t.device != dev \
            or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} "
                         f"on {dev}")


def _ptr(t):
    return None if t is None else t.data_ptr()


def _strides(t):
    """Strides in elements; those of a single entry are never used."""
    return [st if n > 1 else 0 for st, n in zip(t.stride(), t.shape)]


def _rows(name, t, shape, dtype, dev):
    if not isinstance(t, torch.Tensor) or t.shape != shape or t.dtype != dtype or t.device != dev \
            or t.stride(-1) != 1:
        raise ValueError(f"{name} must be a {dtype} tensor of shape {tuple(shape)} on {dev} whose "
                         "last dimension is contiguous")
    b, n, h, _ = _strides(t)
    return RowsArg(t.data_ptr(), b, n, h)


def _cache(k_cache, v_cache, page_table, cache_lens, layered=False):
    """The cache argument, with B."""
    if k_cache.dim() not in ((4, 5) if layered else (4,)):
        raise ValueError("k_cache must be [pages, page_size, heads, head_dim]"
                         + (" or [layers, pages, page_size, heads, head_dim]" if layered else ""))
    if k_cache.dtype not in _CACHE_DTYPES:
        raise TypeError(f"k_cache must be bfloat16 or float16, got {k_cache.dtype}")
    dev = k_cache.device
    st = _strides(k_cache)
    if v_cache.shape != k_cache.shape or v_cache.dtype != k_cache.dtype or v_cache.device != dev \
            or _strides(v_cache) != st or k_cache.stride(-1) != 1:
        raise ValueError("v_cache must have k_cache's shape, strides, type and device, and both a "
                         "contiguous last dimension")
    if page_table.dim() != 2 or page_table.dtype != torch.int32 or page_table.device != dev \
            or (page_table.stride(1) != 1 and page_table.shape[1] > 1):
        raise ValueError(f"page_table must be an int32 tensor [B, pages of a request] on {dev} with "
                         "contiguous rows")
    B, max_pages = page_table.shape
    _need("cache_lens", cache_lens, (B,), torch.int32, dev)
    layers, layer_stride = (k_cache.shape[0], st[0]) if k_cache.dim() == 5 else (1, 0)
    pages, page_size, heads, head_dim = k_cache.shape[-4:]
    return CacheArg(k_cache.data_ptr(), v_cache.data_ptr(), page_table.data_ptr(),
                    cache_lens.data_ptr(), layer_stride, st[-4], st[-3], st[-2], layers, pages,
                    page_size, max_pages, page_table.stride(0) if B > 1 else max_pages, heads,
                    head_dim, _CACHE_DTYPES[k_cache.dtype]), B


def _tree(parents, n_nodes, B, N, dev):
    if parents is not None:
        _need("parents", parents, (B, N), torch.int32, dev)
    if n_nodes is not None:
        _need("n_nodes", n_nodes, (B,), torch.int32, dev)


def _status(status, B, dev):
    if status is None:
        return torch.empty(B, dtype=torch.int32, device=dev)
    _need("status", status, (B,), torch.int32, dev)
    return status


def _nodes_of(q):
    if q.dim() != 4:
        raise ValueError("q must be [B, N, q_heads, head_dim]")
    return q.shape


def append_nodes(q, k, v, k_cache, v_cache, page_table, cache_lens, inv_freq=None, parents=None,
                 n_nodes=None, *, q_weight=None, k_weight=None, eps=1e-6, interleaved=False,
                 rope_scale=1.0, q_out=None, status=None, stream=None):
    """Norms, rotates and appends the projections of a drafted tree's nodes.

    q [B, N, q_heads, D], k and v [B, N, heads, D] bf16 or f16 (views of one
    projection will do); k_cache, v_cache [pages, page_size, heads, D];
    page_table [B, P] and cache_lens [B] int32.  Each head of q and k is
    divided by the root of its mean square plus ``eps`` and multiplied by
    ``q_weight`` / ``k_weight`` [D] (None: no norm), then its first
    2 * len(inv_freq) elements are rotated by (cache_lens[b] + depth of the
    node) * ``inv_freq`` (f32; None: no rotation), in pairs (2j, 2j + 1) if
    ``interleaved`` and (j, j + len(inv_freq)) if not, and scaled by
    ``rope_scale``.  Node i's key and value go to cache slot
    cache_lens[b] + i.  ``parents`` [B, N] int32 (None: a chain), ``n_nodes``
    [B] int32 (None: all N).  Returns (q_out, status [B] int32: 0 or DEV_*
    bits); rows of q_out behind n_nodes[b] are left as they were (zeros in a
    new one).  ``q_out`` may be q.  Asynchronous."""
    B, N, Hq, D = _nodes_of(q)
    cache, rows = _cache(k_cache, v_cache, page_table, cache_lens)
    dev, dtype = k_cache.device, k_cache.dtype
    if rows != B or cache.head_dim != D:
        raise ValueError(f"q is for {B} requests and heads of {D}, the cache for {rows} and "
                         f"{cache.head_dim}")
    q_arg = _rows("q", q, (B, N, Hq, D), dtype, dev)
    k_arg = _rows("k", k, (B, N, cache.heads, D), dtype, dev)
    v_arg = _rows("v", v, (B, N, cache.heads, D), dtype, dev)
    _tree(parents, n_nodes, B, N, dev)
    for name, weight in (("q_weight", q_weight), ("k_weight", k_weight)):
        if weight is not None:
            _need(name, weight, (D,), dtype, dev)
    half = 0
    if inv_freq is not None:
        half = inv_freq.numel()
        _need("inv_freq", inv_freq, (half,), torch.float32, dev)
    with _on(dev, stream):
        if q_out is None:
            q_out = (torch.empty if n_nodes is None else torch.zeros)(B, N, Hq, D, dtype=dtype,
                                                                      device=dev)
        out_arg = _rows("q_out", q_out, (B, N, Hq, D), dtype, dev)
        status = _status(status, B, dev)
        check("spec_append_nodes", lib().spec_append_nodes(
            cache, q_arg, k_arg, v_arg, _ptr(parents), _ptr(n_nodes), B, N, Hq, _ptr(q_weight),
            _ptr(k_weight), eps, _ptr(inv_freq) if half else None, 2 * half, int(interleaved),
            rope_scale, out_arg, status.data_ptr(), _current(dev)))
    return q_out, status


class AttentionWorkspace:
    """Device workspace for tree_attention over B requests of up to N nodes.
    It keeps nothing between calls; calls that may run at the same time (on
    two streams, or two captured graphs that may be replayed together) need
    one each."""

    def __init__(self, B: int, N: int, q_heads: int, kv_heads: int, head_dim: int, device=None):
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
    B, N, Hq, D = _nodes_of(q)
    cache, rows = _cache(k_cache, v_cache, page_table, cache_lens)
    dev, dtype = k_cache.device, k_cache.dtype
    if rows != B or cache.head_dim != D or Hq % cache.heads:
        raise ValueError(f"q is for {B} requests and {Hq} heads of {D}, the cache for {rows} and "
                         f"{cache.heads} of {cache.head_dim}")
    q_arg = _rows("q", q, (B, N, Hq, D), dtype, dev)
    _tree(parents, n_nodes, B, N, dev)
    with _on(dev, stream):
        if out is None:
            out = (torch.empty if n_nodes is None else torch.zeros)(B, N, Hq, D, dtype=dtype,
                                                                    device=dev)
        out_arg = _rows("out", out, (B, N, Hq, D), dtype, dev)
        status = _status(status, B, dev)
        if workspace is None:
            workspace = AttentionWorkspace(B, N, Hq, cache.heads, D, device=dev)
        elif workspace.tensor.device != dev:
            raise ValueError(f"workspace is on {workspace.tensor.device}, the cache on {dev}")
        check("spec_tree_attention", lib().spec_tree_attention(
            cache, q_arg, _ptr(parents), _ptr(n_nodes), B, N, Hq,
            1.0 / math.sqrt(D) if scale is None else scale, out_arg, status.data_ptr(),
            workspace.tensor.data_ptr(), workspace.nbytes, _current(dev)))
    return out, status


def keep_path(path_nodes, accepted_len, k_cache, v_cache, page_table, cache_lens, *, new_lens=None,
              status=None, stream=None):
    """Keeps the accepted path's rows of the cache: slot cache_lens[b] + j gets
    the row of slot cache_lens[b] + path_nodes[b, j], j = 1 ..
    accepted_len[b] (the outputs of verify_tree_greedy).  k_cache and v_cache
    may be [layers, pages, page_size, heads, D]: every layer in one call.
    Returns (new_lens [B] = cache_lens + accepted_len + 1, status [B]) int32;
    a flagged request keeps its rows and its length.  Asynchronous."""
    cache, B = _cache(k_cache, v_cache, page_table, cache_lens, layered=True)
    dev = k_cache.device
    if path_nodes.dim() != 2:
        raise ValueError("path_nodes must be [B, N]")
    N = path_nodes.shape[1]
    _need("path_nodes", path_nodes, (B, N), torch.int32, dev)
    _need("accepted_len", accepted_len, (B,), torch.int32, dev)
    with _on(dev, stream):
        if new_lens is None:
            new_lens = torch.empty(B, dtype=torch.int32, device=dev)
        _need("new_lens", new_lens, (B,), torch.int32, dev)
        status = _status(status, B, dev)
        check("spec_keep_path", lib().spec_keep_path(
            cache, path_nodes.data_ptr(), accepted_len.data_ptr(), B, N, new_lens.data_ptr(),
            status.data_ptr(), _current(dev)))
    return new_lens, status


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
    if logits.dim() not in (2, 3):
        raise ValueError("logits must be [B, R, V] or [B, V]")
    if logits.dtype not in _LOGIT_DTYPES:
        raise TypeError(f"logits must be bfloat16 or float32, got {logits.dtype}")
    given, shape = logits, logits.shape
    B, V = shape[0], shape[-1]
    R = shape[1] if logits.dim() == 3 else 1
    dev, dtype = logits.device, logits.dtype
    if history.dim() != 2 or history.dtype != torch.int32 or history.device != dev \
            or history.shape[0] != B or (history.stride(1) != 1 and history.shape[1] > 1):
        raise ValueError(f"history must be an int32 tensor [B, L] on {dev} with contiguous rows")
    _need("seq_lens", seq_lens, (B,), torch.int32, dev)
    _tree(parents, n_nodes, B, R, dev)
    if tokens is not None:
        _need("tokens", tokens, (B, R if parents is not None else R - 1), torch.int32, dev)
    elif R > 1:
        raise ValueError("tokens must be given for more than one row")
    if prompt_lens is not None:
        _need("prompt_lens", prompt_lens, (B,), torch.int32, dev)
    for name, t in (("repetition", repetition), ("frequency", frequency), ("presence", presence)):
        if t is not None:
            _need(name, t, (B,), torch.float32, dev)
    if (bias_tokens is None) != (bias_values is None):
        raise ValueError("bias_tokens and bias_values go together")
    num_bias = 0
    if bias_tokens is not None:
        num_bias = bias_tokens.shape[-1]
        _need("bias_tokens", bias_tokens, (B, num_bias), torch.int32, dev)
        _need("bias_values", bias_values, (B, num_bias), torch.float32, dev)
    if allowed is not None:
        _need("allowed", allowed, shape[:-1] + (-(-V // 32),), torch.int32, dev)

    def rows(name, t):
        if t.shape != shape or t.dtype != dtype or t.device != dev or (V > 1 and t.stride(-1) != 1):
            raise ValueError(f"{name} must be a {dtype} tensor of shape {tuple(shape)} on {dev} whose "
                             "last dimension is contiguous")
        st = _strides(t)
        return st[0], st[1] if t.dim() == 3 else 0

    in_strides = rows("logits", given)
    with _on(dev, stream):
        if out is None:
            out = (torch.empty if n_nodes is None else torch.zeros)(shape, dtype=dtype, device=dev)
        out_strides = rows("out", out)
        status = _status(status, B, dev)
        check("spec_process_logits", lib().spec_process_logits(
            logits.data_ptr(), *in_strides, _LOGIT_DTYPES[dtype], B, R, V,
            _ptr(tokens) if R > 1 else None, _ptr(parents), _ptr(n_nodes), history.data_ptr(),
            history.stride(0) if B > 1 else 0, history.shape[1], seq_lens.data_ptr(),
            _ptr(prompt_lens), _ptr(repetition), _ptr(frequency), _ptr(presence),
            _ptr(bias_tokens), _ptr(bias_values), num_bias, _ptr(allowed), out.data_ptr(),
            *out_strides, status.data_ptr(), _current(dev)))
    return out, status
