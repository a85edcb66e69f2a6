"""The operators before the verification without a GPU: what the entry points
refuse before they touch the device."""

import struct

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import prompt_reference as ref  # noqa: E402
import speculative_decoding_verify_sample_gb300 as sv  # noqa: E402
from test_chunk_items_cpu import run as run_on_host  # noqa: E402
from test_tree_cpu import BAD_CACHES, FAKE, INVALID, UNSUPPORTED, cache  # noqa: E402


@pytest.fixture(scope="module")
def L():
    sv.build()
    return sv.lib()


def rows(data=FAKE, t=64 * 8, h=64):
    return struct.pack("@P3q", data or 0, 0, t, h)  # specv_rows, packed


def append(L, c=None, **over):
    a = dict(cache=c or cache(), q=rows(), k=rows(), v=rows(), cu=FAKE, B=2, T=40, heads=4, pos=FAKE,
             ps=40, axes=3, axis=FAKE, qw=FAKE, kw=FAKE, eps=1e-6, inv=FAKE, rot=64, inter=0, scale=1.0,
             out=rows(), status=FAKE)
    a.update(over)
    return L.spec_append_chunk(*a.values(), None)


def attend(L, c=None, **over):
    a = dict(cache=c or cache(), q=rows(), cu=FAKE, B=2, T=40, longest=30, heads=4, scale=0.1, cap=0.0,
             window=0, prefix=FAKE, slopes=FAKE, out=rows(), status=FAKE, ws=FAKE, bytes=1 << 40)
    a.update(over)
    return L.spec_chunk_attention(*a.values(), None)


def select(L, **over):
    a = dict(z=FAKE, bs=400, rs=100, dtype=1, B=2, W=4, V=100, K=4, scores=FAKE, ended=FAKE, end=0,
             out=FAKE, tokens=FAKE, beams=FAKE, status=FAKE, ws=FAKE, bytes=1 << 40)
    a.update(over)
    return L.spec_select_beams(*a.values(), None)


def state(i=FAKE, o=2 * FAKE, ib=400, iw=100, ob=400, ow=100, n=100):
    return struct.pack("@2P5q", i or 0, o or 0, ib, iw, ob, ow, n)  # specv_state


def reorder(L, **over):
    a = dict(beams=FAKE, B=2, W=4, K=4, states=state(), num=1, status=FAKE)
    a.update(over)
    return L.spec_reorder_beams(*a.values(), None)


@pytest.mark.parametrize("call", [append, attend])
def test_cache_limits(L, call):
    for over, status in BAD_CACHES:
        assert call(L, cache(**over)) == status, over
    assert call(L, B=0) == INVALID
    assert call(L, B=65536) == UNSUPPORTED
    assert call(L, cache(layers=2)) == INVALID


@pytest.mark.parametrize("over,status", [
    (dict(q=rows(None)), 1), (dict(k=rows(FAKE + 8)), 1), (dict(v=rows(t=4)), 1), (dict(out=rows(h=63)), 1),
    (dict(q=None), 1), (dict(status=None), 1), (dict(cu=None), 1), (dict(cu=FAKE + 2), 1), (dict(T=-1), 1),
    (dict(heads=0), 1), (dict(heads=1025), 2), (dict(rot=63), 1), (dict(rot=66), 1), (dict(rot=0), 1),
    (dict(inv=None), 1), (dict(axes=0), 1), (dict(ps=39), 1), (dict(ps=-1), 1), (dict(axis=None), 1),
    (dict(pos=None), 1), (dict(pos=FAKE + 2), 1), (dict(axis=FAKE + 1), 1), (dict(eps=-1.0), 1),
    (dict(eps=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(qw=FAKE + 2), 1),
    (dict(kw=FAKE + 8), 1), (dict(status=FAKE + 2), 1), (dict(inv=FAKE + 2), 1),
])
def test_append_refusals(L, over, status):
    assert append(L, **over) == status


@pytest.mark.parametrize("over,status", [
    (dict(q=rows(None)), 1), (dict(out=rows(FAKE + 4)), 1), (dict(out=None), 1), (dict(q=rows(t=12)), 1),
    (dict(status=None), 1), (dict(ws=None), 1), (dict(ws=FAKE + 128), 1), (dict(bytes=16), 3),
    (dict(cu=None), 1), (dict(cu=FAKE + 1), 1), (dict(T=-1), 1), (dict(longest=0), 1), (dict(heads=3), 1),
    (dict(heads=0), 1), (dict(heads=1026), 2), (dict(scale=0.0), 1), (dict(scale=-1.0), 1),
    (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(cap=-1.0), 1),
    (dict(cap=float("nan")), 1), (dict(cap=float("inf")), 1), (dict(cap=1e-38), 1), (dict(window=-1), 1),
    (dict(prefix=FAKE + 2), 1), (dict(slopes=FAKE + 2), 1), (dict(status=FAKE + 1), 1),
    (dict(B=16385), 2), (dict(longest=2 ** 29), 2),
])
def test_attention_refusals(L, over, status):
    assert attend(L, **over) == status


@pytest.mark.parametrize("over,status", [
    (dict(z=None), 1), (dict(scores=None), 1), (dict(out=None), 1), (dict(tokens=None), 1),
    (dict(beams=None), 1), (dict(status=None), 1), (dict(ws=None), 1), (dict(ws=FAKE + 64), 1),
    (dict(bytes=8), 3), (dict(dtype=2), 1), (dict(B=0), 1), (dict(W=0), 1), (dict(K=0), 1), (dict(V=0), 1),
    (dict(bs=-1), 1), (dict(rs=-2), 1), (dict(z=FAKE + 1), 1), (dict(dtype=0, z=FAKE + 2), 1),
    (dict(scores=FAKE + 2), 1), (dict(ended=FAKE + 1), 1), (dict(tokens=FAKE + 2), 1),
    (dict(W=65), 2), (dict(K=65), 2), (dict(B=65536), 2), (dict(V=1048577), 2), (dict(dtype=0, V=524289), 2),
])
def test_select_refusals(L, over, status):
    assert select(L, **over) == status


@pytest.mark.parametrize("over,status", [
    (dict(beams=None), 1), (dict(states=None), 1), (dict(status=None), 1), (dict(num=0), 1), (dict(num=33), 2),
    (dict(beams=FAKE + 2), 1), (dict(status=FAKE + 1), 1), (dict(B=0), 1), (dict(W=0), 1), (dict(K=0), 1),
    (dict(W=65), 2), (dict(K=65), 2), (dict(B=65536), 2), (dict(states=state(None)), 1),
    (dict(states=state(o=None)), 1), (dict(states=state(n=0)), 1), (dict(states=state(iw=-1)), 1),
    (dict(states=state(ow=99)), 1), (dict(states=state(o=FAKE, ow=200)), 1),
    (dict(states=state(o=FAKE, ob=800)), 1), (dict(states=state(n=2 ** 40, ow=2 ** 40)), 2),
])
def test_reorder_refusals(L, over, status):
    assert reorder(L, **over) == status


def test_reorder_refuses_states_on_one_another(L):
    """Written twice, or read and written by different states, or moved onto part of itself."""
    a = dict(ib=48, iw=10, ob=48, ow=10, n=8)
    for off in (-8, 0, 4, 8, 14, 54, 60):  # (the beams' gaps have 2 bytes)
        for two in (state(o=8 * FAKE, **a) + state(2 * FAKE, 8 * FAKE + off, **a),
                    state(o=8 * FAKE, **a) + state(2 * FAKE, FAKE + off, **a)):
            assert reorder(L, states=two, num=2) == INVALID, off
        if off:
            assert reorder(L, states=state(o=FAKE + off, **a)) == INVALID, off
    for other in (dict(a, ow=20), dict(a, ob=96)):  # other strides: where both begin together
        assert reorder(L, states=state(o=8 * FAKE, **a) + state(2 * FAKE, 8 * FAKE, **other), num=2) == INVALID


PLACES = r"""
#include <cstdio>
#include <set>
#include "beams.cu"

int specv_max_vocab(specv_dtype) { return 0; }  // (of another file; not called)

int main() {
  int met = 0, apart = 0;
  for (int B : {1, 2, 3})
    for (int W : {1, 3})
      for (int K : {1, 2, 3})
        for (int batch : {0, 7, 16, 40})
          for (int beam : {0, 3, 7, 40})
            for (int n : {1, 3, 5})
              for (int off = -130; off <= 130; off++) {
                const auto place = [](int at) { return reinterpret_cast<const void*>(static_cast<uintptr_t>(at)); };
                const Places x(place(1000), batch, beam, n, B, W), y(place(1000 + off), batch, beam, n + 1, B, K);
                std::set<int> bytes;
                bool want = false;
                for (int b = 0; b < B; b++)
                  for (int w = 0; w < W; w++)
                    for (int e = 0; e < n; e++) bytes.insert(1000 + b * batch + w * beam + e);
                for (int b = 0; b < B; b++)
                  for (int k = 0; k < K; k++)
                    for (int e = 0; e <= n; e++) want |= bytes.count(1000 + off + b * batch + k * beam + e) > 0;
                if (overlap(x, y) != want || overlap(y, x) != want) {
                  std::printf("B %d W %d K %d batch %d beam %d n %d off %d: not %d\n", B, W, K, batch, beam, n, off, want);
                  return 1;
                }
                (want ? met : apart)++;
              }
  std::printf("%d\n", met < apart ? met : apart);
}
"""


def test_reorder_knows_which_places_meet(tmp_path):
    """Against all bytes of both, for strides that are alike."""
    assert int(run_on_host(PLACES, tmp_path)) > 10000


def test_workspace_sizes(L):
    assert L.specv_chunk_workspace_bytes(0, 8, 8, 64) == 0
    assert L.specv_chunk_workspace_bytes(4, 9, 8, 64) == 0
    assert L.specv_chunk_workspace_bytes(4, 8, 8, 60) == 0
    assert L.specv_chunk_workspace_bytes(2 ** 29, 8, 8, 64) == 0
    few, many = (L.specv_chunk_workspace_bytes(n, 8, 8, 64) for n in (1, 4096))
    assert 0 < few < many
    assert many == L.specv_chunk_workspace_bytes(1 << 20, 8, 8, 64)  # however long
    assert L.specv_beam_workspace_bytes(0, 1, 1, 10) == 0
    assert L.specv_beam_workspace_bytes(1, 65, 1, 10) == 0
    assert L.specv_beam_workspace_bytes(1, 1, 65, 10) == 0
    assert L.specv_beam_workspace_bytes(1, 1, 1, (1 << 20) + 1) == 0
    assert L.specv_beam_workspace_bytes(2, 8, 8, 128256) > 2 * 8 * 8 * 8
    with pytest.raises(ValueError):
        sv.ChunkWorkspace(4, 9, 8, 64)
    with pytest.raises(ValueError):
        sv.BeamWorkspace(1, 65, 1, 10)


def test_a_beam_workspace_serves_smaller_calls(L):
    """What is enough for a call is enough for one of fewer requests, beams, places or entries."""
    need = L.specv_beam_workspace_bytes
    for W, K, V in ((8, 8, 128256), (1, 1, 9), (5, 3, 32003), (64, 64, 50000), (2, 17, 1 << 20)):
        sizes = [need(B, W, K, V) for B in (*range(1, 600), 4000, 65535)]
        assert sizes[0] > 0 and sizes == sorted(sizes), (W, K, V)
    for B in (1, 3, 40, 64, 700):
        sizes = [need(B, W, 8, 128256) for W in range(1, 65)]
        assert sizes == sorted(sizes), B
        sizes = [need(B, 8, K, 128256) for K in range(1, 65)]
        assert sizes == sorted(sizes), B
        sizes = [need(B, 8, 8, V) for V in (*range(1, 140000, 511), 131072, 131073, 1 << 20)]
        assert sizes[:-3] == sorted(sizes[:-3]) and sizes[-3] <= sizes[-2] <= sizes[-1], B


PLANS = r"""
#include <cstdio>
#include "beams.cu"

int specv_max_vocab(specv_dtype) { return 0; }  // (of another file; not called)

int main() {
  int calls = 0;
  for (int B = 1; B <= 600; B += B < 100 ? 1 : 7)
    for (int W : {1, 2, 5, 8, 31, 64})
      for (int K : {1, 8, 64})
        for (int V : {1, 4095, 4096, 4097, 8193, 32003, 50000, 128256, 131072, 131073, 524288, 1 << 20}) {
          const size_t most = specv_beam_workspace_bytes(B, W, K, V);
          const size_t half = Plan(B, W, K, V, kStepOf<SPECV_BF16>).total;
          const size_t full = Plan(B, W, K, V, kStepOf<SPECV_F32>).total;
          if (half > most || full > most) {
            std::printf("B %d W %d K %d V %d: %zu, needed %zu and %zu\n", B, W, K, V, most, half, full);
            return 1;
          }
          calls++;
        }
  std::printf("%d\n", calls);
}
"""


def test_a_beam_workspace_is_large_enough(tmp_path):
    assert int(run_on_host(PLANS, tmp_path)) > 10000


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def prompt_args(T=6, Hq=4, Hkv=2, D=64, dtype=torch.bfloat16):
    cache = torch.zeros(3, 16, Hkv, D, dtype=dtype)
    q, k = torch.zeros(T, Hq, D, dtype=dtype), torch.zeros(T, Hkv, D, dtype=dtype)
    return q, k, cache, i32(2, 2), i32(2), i32(3)


def test_binding_refuses_wrong_arguments():
    """Wrong shapes, types and places by name; CPU tensors last, when all else is right."""
    q, k, cache, table, lens, cu = prompt_args()

    def attend(q=q, cu=cu, **kw):
        return sv.chunk_attention(q, cache, cache.clone(), table, lens, cu, **kw)

    def append(q=q, k=k, v=k, cu=cu, freq=torch.ones(32), **kw):
        return sv.append_chunk(q, k, v, cache, cache.clone(), table, lens, cu, freq, **kw)

    for call in (attend, append):
        with pytest.raises(ValueError, match="CUDA tensors"):
            call()
        with pytest.raises(ValueError, match="cu_tokens"):
            call(cu=i32(2))
        with pytest.raises(ValueError, match="cu_tokens"):
            call(cu=None)
        with pytest.raises(ValueError, match="q must be"):
            call(q=q[None])
        with pytest.raises(ValueError, match="q must be"):
            call(q=q.half())
    for kw, what in [(dict(cap=0.0), "cap"), (dict(cap=-2.0), "cap"), (dict(window=0), "window"),
                     (dict(longest=0), "longest"), (dict(prefix_lens=i32(3)), "prefix_lens"),
                     (dict(slopes=torch.ones(3)), "slopes"), (dict(window=2 ** 40), "window")]:
        with pytest.raises(ValueError, match=what):
            attend(**kw)
    with pytest.raises(ValueError, match="heads"):
        attend(q=torch.zeros(6, 5, 64, dtype=q.dtype))
    for kw, what in [(dict(positions=i32(3, 5)), "positions"), (dict(positions=i32(3, 6)), "axis_of"),
                     (dict(axis_of=i32(32)), "axis_of"), (dict(positions=i32(3, 6), axis_of=i32(31)), "axis_of"),
                     (dict(positions=i32(1, 6).expand(3, 6), axis_of=i32(32)), "positions"),
                     (dict(q_weight=torch.ones(64)), "q_weight"), (dict(k=k[:5]), "k must be"),
                     (dict(freq=torch.ones(32).half()), "inv_freq")]:
        with pytest.raises(ValueError, match=what):
            append(**kw)

    z, scores = torch.zeros(2, 3, 50), torch.zeros(2, 3)
    with pytest.raises(ValueError, match="CUDA tensors"):
        sv.select_beams(z, scores)
    with pytest.raises(TypeError):
        sv.select_beams(z.half(), scores)
    for kw, what in [(dict(width=0), "width"), (dict(ended=i32(2)), "ended"), (dict(beams=i32(2, 4)), "beams"),
                     (dict(end_token=2 ** 40), "end_token")]:
        with pytest.raises(ValueError, match=what if "beams" not in kw else "CUDA tensors"):
            sv.select_beams(z, scores, **kw)
    with pytest.raises(ValueError, match="logits"):
        sv.select_beams(z[0], scores)
    with pytest.raises(ValueError, match="scores"):
        sv.select_beams(z, scores.double())
    with pytest.raises(ValueError, match="last dimension"):
        sv.select_beams(z.transpose(1, 2).contiguous().transpose(1, 2), scores)

    beams, state = i32(2, 3), torch.zeros(2, 3, 7)
    with pytest.raises(ValueError, match="CUDA tensors"):
        sv.reorder_beams(beams, state)
    for states, out, what in [([], None, "one tensor or more"), ([state, state[:, :2]], None, "one W"),
                              (state, torch.zeros(2, 3, 8), "out"), (state, torch.zeros(2, 4, 7), "out"),
                              (torch.zeros(2, 4, 7), None, "out"), (state[:, :, ::2], None, "contiguous"),
                              (state, state[:, :1].expand(2, 3, 7), "every element"),
                              (state, [state, state], "as many out"), (state.double(), state, "out")]:
        with pytest.raises(ValueError, match=what):
            sv.reorder_beams(beams, states, out=out)


def test_plain_attention_is_the_masked_softmax():
    """The plain form that the GPU tests compare with, against a dense masked softmax."""
    gen = torch.Generator().manual_seed(1)
    T, Hq, Hkv, D, page = 9, 4, 2, 8, 4
    lens, cu = [5, 0, 3], [0, 4, 4, 9]
    k, v = (torch.randn(8, page, Hkv, D, generator=gen) for _ in "kv")
    table = torch.tensor([[0, 1, 2], [7, 7, 7], [3, 4, 5]], dtype=torch.int32)
    q = torch.randn(T, Hq, D, generator=gen)
    slopes = torch.tensor([0.5, 0.25, 0.125, 0.0])
    for cap, window, prefix, bias in [(None, None, None, None), (5.0, 3, None, None), (None, 2, [3, 0, 99], slopes)]:
        out, tol = ref.attention(q, k, v, table, lens, cu, 0.3, cap, window, prefix, bias)
        assert torch.isfinite(out).all() and (tol > 0).all()
        for b in range(3):
            for t in range(cu[b], cu[b + 1]):
                p = lens[b] + t - cu[b]
                for h in range(Hq):
                    w, total = torch.zeros(D, dtype=torch.float64), 0.0
                    for s in range(lens[b] + cu[b + 1] - cu[b]):
                        inside = prefix is not None and s < prefix[b]
                        if not inside and (s > p or (window and p - s >= window)):
                            continue
                        row = k[table[b, s // page].long(), s % page, h // 2].double()
                        y = float(q[t, h].double() @ row) * 0.3
                        y = cap * np.tanh(y / cap) if cap else y
                        y -= float(bias[h]) * abs(p - s) if bias is not None else 0.0
                        total += np.exp(y)
                        w += np.exp(y) * v[table[b, s // page].long(), s % page, h // 2].double()
                    assert torch.allclose(out[t, h], w / total, rtol=1e-9, atol=1e-12)
