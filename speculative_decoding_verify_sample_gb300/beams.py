"""Binding of the drafting of a tree level by level, or a beam search: the best
next tokens of all beams, and the beams' states moved along ("Accelerating Sonar
through speculation", section "EAGLE": a tree of candidates from the draft's own
probabilities).

Shapes, types and devices are checked in csrc/binding.cpp, limits in the library;
every step runs in its kernels.
"""

from __future__ import annotations

from . import tree
from ._native import lib


class BeamWorkspace:
    """Device workspace for select_beams of up to K among up to W beams of vocabularies of
    up to V entries, for up to B requests.  Calls that may run at the same time need one each."""

    def __init__(self, B: int, W: int, K: int, V: int, device=None):
        import torch
        self.nbytes = int(lib().specv_beam_workspace_bytes(B, W, K, V))
        if self.nbytes == 0:
            raise ValueError(f"unsupported beam shape B={B} W={W} K={K} V={V}")
        self.tensor = torch.empty(self.nbytes, dtype=torch.uint8, device=device)


def select_beams(logits, scores, width=None, *, ended=None, end_token=0, out_scores=None,
                 tokens=None, beams=None, status=None, workspace=None, stream=None):
    """The ``width`` (None: W) best next tokens of each request's W beams.

    logits [B, W, V] bf16 or f32: what the model says after each beam; scores
    [B, W] f32: its summed log probability (-inf: not in play).  Of all beams w
    and tokens v the largest scores[b, w] + log softmax(logits[b, w])[v], falling,
    ties to the lower beam and then the lower token: the nodes of a drafted
    tree's next level, or a beam search's step.  A beam with ``ended`` [B, W]
    int32 not 0 is one candidate, with the score that it has and ``end_token``.
    Returns (out_scores [B, width] f32, tokens, beams [B, width] int32, status
    [B] int32: 0 or DEV_* bits); behind the last candidate -inf, -1, -1.
    Asynchronous."""
    return tree._call("spec_select_beams", (tree._binding or tree.load()).select_beams, logits, stream,
                      logits, scores, width, ended, end_token, out_scores, tokens, beams, status,
                      None if workspace is None else workspace.tensor)


def reorder_beams(beams, states, *, out=None, status=None, stream=None):
    """Moves beams' states to the beams that go on from them: out[b, k] =
    state[b, beams[b, k]].

    ``beams`` [B, K] int32 (select_beams'; -1: the place stays as it was); states:
    a tensor [B, W, ...] of any type, or up to 32 of them (hidden states, texts,
    rows of a page table), each beam's part contiguous: all in one call.
    ``out``: as many tensors [B, K, ...]; None: the states themselves, with K =
    W.  Returns (out, status [B] int32: 0 or DEV_* bits), out a tensor or a tuple
    as the states are; a flagged request's states stay as they were.  No state may be
    given twice, nor lie on memory that another is moved to.
    Asynchronous."""
    one = hasattr(states, "is_cuda")
    given = (states,) if one else tuple(states)
    outs = given if out is None else (out,) if hasattr(out, "is_cuda") else tuple(out)
    status, = tree._call("spec_reorder_beams", (tree._binding or tree.load()).reorder_beams, beams,
                         stream, beams, given, outs, status)
    return (outs[0] if one else outs), status
