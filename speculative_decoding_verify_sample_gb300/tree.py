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
import math
import struct

import torch

from ._native import ATTENTION_HEADER_BYTES, SPECV_BF16, SPECV_F16, SPECV_F32, check, lib

_CACHE_DTYPES = {torch.bfloat16: SPECV_BF16, torch.float16: SPECV_F16}
_LOGIT_DTYPES = {torch.bfloat16: SPECV_BF16, torch.float32: SPECV_F32}
_INT32, _FLOAT32 = torch.int32, torch.float32
# specv_cache and specv_rows of the header, as bytes: these calls take a few
# microseconds on the device, so what the host spends on them counts
_pack_cache = struct.Struct("@4P4q8i").pack
_pack_rows = struct.Struct("@P3q").pack
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _elsewhere(device, stream):
    """Whether the call has to be made on another device or stream than the
    current ones (it allocates on what it launches on)."""
    if device.type != "cuda":
        raise ValueError(f"the operators on a drafted tree take CUDA tensors, got {device}")
    return stream is not None or device.index != torch.cuda.current_device()


@contextlib.contextmanager
def _there(device, stream):
    with torch.cuda.device(device):
        if stream is None:
            yield
        else:
            if not isinstance(stream, torch.cuda.Stream):
                stream = torch.cuda.ExternalStream(getattr(stream, "cuda_stream", stream), device)
            with torch.cuda.stream(stream):
                yield


def _need(name, t, shape, dtype, dev):
    """t is a contiguous tensor of this shape, type and device."""
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.shape != shape or t.device != dev \
            or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} "
                         f"on {dev}")


def _ptr(t):
    return None if t is None else t.data_ptr()


def _strides(t, shape):
    """Strides in elements; those of a single entry are never used."""
    st = t.stride()
    return [s if n > 1 else 0 for s, n in zip(st, shape)] if 1 in shape else st


def _rows(name, t, shape, dtype, dev):
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.shape != shape or t.device != dev:
        raise ValueError(f"{name} must be a {dtype} tensor of shape {tuple(shape)} on {dev}")
    b, n, h, d = _strides(t, shape)
    if d != 1:
        raise ValueError(f"{name} must have a contiguous last dimension")
    return _pack_rows(t.data_ptr(), b, n, h)


def _cache(k_cache, v_cache, page_table, cache_lens, layered=False):
    """(the cache argument, B, heads, head_dim)."""
    shape, dtype, dev = k_cache.shape, k_cache.dtype, k_cache.device
    if len(shape) != 4 and not (layered and len(shape) == 5):
        raise ValueError("k_cache must be [pages, page_size, heads, head_dim]"
                         + (" or [layers, pages, page_size, heads, head_dim]" if layered else ""))
    code = _CACHE_DTYPES.get(dtype)
    if code is None:
        raise TypeError(f"k_cache must be bfloat16 or float16, got {dtype}")
    st = _strides(k_cache, shape)
    if v_cache.shape != shape or v_cache.dtype != dtype or v_cache.device != dev \
            or _strides(v_cache, shape) != st or st[-1] != 1:
        raise ValueError("v_cache must have k_cache's shape, strides, type and device, and both a "
                         "contiguous last dimension")
    if page_table.dim() != 2 or page_table.dtype != _INT32 or page_table.device != dev \
            or (page_table.stride(1) != 1 and page_table.shape[1] > 1):
        raise ValueError(f"page_table must be an int32 tensor [B, pages of a request] on {dev} with "
                         "contiguous rows")
    B, max_pages = page_table.shape
    _need("cache_lens", cache_lens, (B,), _INT32, dev)
    pages, page_size, heads, head_dim = shape[-4:]
    layers, layer_stride = (shape[0], st[0]) if len(shape) == 5 else (1, 0)
    return _pack_cache(k_cache.data_ptr(), v_cache.data_ptr(), page_table.data_ptr(),
                       cache_lens.data_ptr(), layer_stride, st[-4], st[-3], st[-2], layers, pages,
                       page_size, max_pages, page_table.stride(0) if B > 1 else max_pages, heads,
                       head_dim, code), B, heads, head_dim


def _tree(parents, n_nodes, B, N, dev):
    if parents is not None:
        _need("parents", parents, (B, N), _INT32, dev)
    if n_nodes is not None:
        _need("n_nodes", n_nodes, (B,), _INT32, dev)


def _per_request(name, t, B, dev):
    """An int32 output [B], made here if the caller gave none."""
    if t is None:
        return torch.empty(B, dtype=_INT32, device=dev)
    _need(name, t, (B,), _INT32, dev)
    return t


def _new(n_nodes, shape, dtype, dev):
    """An output that the caller did not give: zeros where rows may be left."""
    return (torch.empty if n_nodes is None else torch.zeros)(shape, dtype=dtype, device=dev)


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
    cache, rows, heads, head_dim = _cache(k_cache, v_cache, page_table, cache_lens)
    dev, dtype = k_cache.device, k_cache.dtype
    if rows != B or head_dim != D:
        raise ValueError(f"q is for {B} requests and heads of {D}, the cache for {rows} and "
                         f"{head_dim}")
    q_arg = _rows("q", q, q.shape, dtype, dev)
    k_arg = _rows("k", k, (B, N, heads, D), dtype, dev)
    v_arg = _rows("v", v, (B, N, heads, D), dtype, dev)
    _tree(parents, n_nodes, B, N, dev)
    if q_weight is not None:
        _need("q_weight", q_weight, (D,), dtype, dev)
    if k_weight is not None:
        _need("k_weight", k_weight, (D,), dtype, dev)
    half = 0
    if inv_freq is not None:
        half = inv_freq.numel()
        _need("inv_freq", inv_freq, (half,), _FLOAT32, dev)
    if _elsewhere(dev, stream):
        with _there(dev, stream):
            return append_nodes(q, k, v, k_cache, v_cache, page_table, cache_lens, inv_freq, parents,
                                n_nodes, q_weight=q_weight, k_weight=k_weight, eps=eps,
                                interleaved=interleaved, rope_scale=rope_scale, q_out=q_out,
                                status=status)
    if q_out is None:
        q_out = _new(n_nodes, q.shape, dtype, dev)
    out_arg = q_arg if q_out is q else _rows("q_out", q_out, q.shape, dtype, dev)
    status = _per_request("status", status, B, dev)
    check("spec_append_nodes", lib().spec_append_nodes(
        cache, q_arg, k_arg, v_arg, _ptr(parents), _ptr(n_nodes), B, N, Hq, _ptr(q_weight),
        _ptr(k_weight), eps, _ptr(inv_freq) if half else None, 2 * half, 1 if interleaved else 0,
        rope_scale, out_arg, status.data_ptr(), _raw_stream(dev.index)))
    return q_out, status


class AttentionWorkspace:
    """Device workspace for tree_attention over B requests of up to N nodes, its
    header zeroed once on creation (every call leaves it ready for the next).  Calls
    that may run at the same time (on two streams, or two captured graphs that
    may be replayed together) need one each."""

    def __init__(self, B: int, N: int, q_heads: int, kv_heads: int, head_dim: int, device=None,
                 stream=None):
        self.nbytes = int(lib().specv_attention_workspace_bytes(B, N, q_heads, kv_heads, head_dim))
        if self.nbytes == 0:
            raise ValueError(f"unsupported attention shape B={B} N={N} q_heads={q_heads} "
                             f"kv_heads={kv_heads} head_dim={head_dim}")
        self.tensor = torch.empty(self.nbytes, dtype=torch.uint8, device=device)
        dev = self.tensor.device
        with torch.cuda.device(dev):
            check("specv_workspace_init", lib().specv_workspace_init(
                self.tensor.data_ptr(), ATTENTION_HEADER_BYTES,
                _raw_stream(dev.index) if stream is None else getattr(stream, "cuda_stream", stream)))


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
    cache, rows, heads, head_dim = _cache(k_cache, v_cache, page_table, cache_lens)
    dev, dtype = k_cache.device, k_cache.dtype
    if rows != B or head_dim != D or Hq % heads:
        raise ValueError(f"q is for {B} requests and {Hq} heads of {D}, the cache for {rows} and "
                         f"{heads} of {head_dim}")
    q_arg = _rows("q", q, q.shape, dtype, dev)
    _tree(parents, n_nodes, B, N, dev)
    if _elsewhere(dev, stream):
        with _there(dev, stream):
            return tree_attention(q, k_cache, v_cache, page_table, cache_lens, parents, n_nodes,
                                  scale=scale, out=out, status=status, workspace=workspace)
    if out is None:
        out = _new(n_nodes, q.shape, dtype, dev)
    out_arg = _rows("out", out, q.shape, dtype, dev)
    status = _per_request("status", status, B, dev)
    if workspace is None:
        workspace = AttentionWorkspace(B, N, Hq, heads, D, device=dev)
    elif workspace.tensor.device != dev:
        raise ValueError(f"workspace is on {workspace.tensor.device}, the cache on {dev}")
    check("spec_tree_attention", lib().spec_tree_attention(
        cache, q_arg, _ptr(parents), _ptr(n_nodes), B, N, Hq,
        1.0 / math.sqrt(D) if scale is None else scale, out_arg, status.data_ptr(),
        workspace.tensor.data_ptr(), workspace.nbytes, _raw_stream(dev.index)))
    return out, status


def keep_path(path_nodes, accepted_len, k_cache, v_cache, page_table, cache_lens, *, new_lens=None,
              status=None, stream=None):
    """Keeps the accepted path's rows of the cache: slot cache_lens[b] + j gets
    the row of slot cache_lens[b] + path_nodes[b, j], j = 1 ..
    accepted_len[b] (the outputs of verify_tree_greedy).  k_cache and v_cache
    may be [layers, pages, page_size, heads, D]: every layer in one call.
    Returns (new_lens [B] = cache_lens + accepted_len + 1, status [B]) int32;
    a flagged request keeps its rows and its length.  Asynchronous."""
    cache, B, _, _ = _cache(k_cache, v_cache, page_table, cache_lens, layered=True)
    dev = k_cache.device
    if path_nodes.dim() != 2:
        raise ValueError("path_nodes must be [B, N]")
    N = path_nodes.shape[1]
    _need("path_nodes", path_nodes, (B, N), _INT32, dev)
    _need("accepted_len", accepted_len, (B,), _INT32, dev)
    if _elsewhere(dev, stream):
        with _there(dev, stream):
            return keep_path(path_nodes, accepted_len, k_cache, v_cache, page_table, cache_lens,
                             new_lens=new_lens, status=status)
    new_lens = _per_request("new_lens", new_lens, B, dev)
    status = _per_request("status", status, B, dev)
    check("spec_keep_path", lib().spec_keep_path(
        cache, path_nodes.data_ptr(), accepted_len.data_ptr(), B, N, new_lens.data_ptr(),
        status.data_ptr(), _raw_stream(dev.index)))
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
    shape, dtype, dev = logits.shape, logits.dtype, logits.device
    B, V = shape[0], shape[-1]
    R = shape[1] if len(shape) == 3 else 1
    if history.dim() != 2 or history.dtype != _INT32 or history.device != dev \
            or history.shape[0] != B or (history.stride(1) != 1 and history.shape[1] > 1):
        raise ValueError(f"history must be an int32 tensor [B, L] on {dev} with contiguous rows")
    _need("seq_lens", seq_lens, (B,), _INT32, dev)
    _tree(parents, n_nodes, B, R, dev)
    if tokens is not None:
        _need("tokens", tokens, (B, R if parents is not None else R - 1), _INT32, dev)
    elif R > 1:
        raise ValueError("tokens must be given for more than one row")
    if prompt_lens is not None:
        _need("prompt_lens", prompt_lens, (B,), _INT32, dev)
    if repetition is not None:
        _need("repetition", repetition, (B,), _FLOAT32, dev)
    if frequency is not None:
        _need("frequency", frequency, (B,), _FLOAT32, dev)
    if presence is not None:
        _need("presence", presence, (B,), _FLOAT32, dev)
    if (bias_tokens is None) != (bias_values is None):
        raise ValueError("bias_tokens and bias_values go together")
    num_bias = 0
    if bias_tokens is not None:
        num_bias = bias_tokens.shape[-1]
        _need("bias_tokens", bias_tokens, (B, num_bias), _INT32, dev)
        _need("bias_values", bias_values, (B, num_bias), _FLOAT32, dev)
    if allowed is not None:
        _need("allowed", allowed, shape[:-1] + (-(-V // 32),), _INT32, dev)

    def rows(name, t):
        if t.shape != shape or t.dtype != dtype or t.device != dev:
            raise ValueError(f"{name} must be a {dtype} tensor of shape {tuple(shape)} on {dev}")
        st = _strides(t, shape)
        if V > 1 and st[-1] != 1:
            raise ValueError(f"{name} must have a contiguous last dimension")
        return st[0], st[1] if R > 1 else 0

    batch_stride, row_stride = rows("logits", logits)
    if _elsewhere(dev, stream):
        with _there(dev, stream):
            return process_logits(logits, history, seq_lens, prompt_lens, tokens=tokens,
                                  parents=parents, n_nodes=n_nodes, repetition=repetition,
                                  frequency=frequency, presence=presence, bias_tokens=bias_tokens,
                                  bias_values=bias_values, allowed=allowed, out=out, status=status)
    if out is None:
        out = _new(n_nodes, shape, dtype, dev)
    out_batch_stride, out_row_stride = rows("out", out)
    status = _per_request("status", status, B, dev)
    check("spec_process_logits", lib().spec_process_logits(
        logits.data_ptr(), batch_stride, row_stride, _LOGIT_DTYPES[dtype], B, R, V,
        _ptr(tokens) if R > 1 else None, _ptr(parents), _ptr(n_nodes), history.data_ptr(),
        history.stride(0) if B > 1 else 0, history.shape[1], seq_lens.data_ptr(), _ptr(prompt_lens),
        _ptr(repetition), _ptr(frequency), _ptr(presence), _ptr(bias_tokens), _ptr(bias_values),
        num_bias, _ptr(allowed), out.data_ptr(), out_batch_stride, out_row_stride, status.data_ptr(),
        _raw_stream(dev.index)))
    return out, status
