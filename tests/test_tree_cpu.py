"""The operators on a drafted tree without a GPU: what the entry points refuse
before they touch the device, and the plain forms the GPU tests compare with."""

import os
import struct
import subprocess
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verify_sample_gb300 as sv  # noqa: E402
import tree_reference as ref  # noqa: E402

FAKE = 0x10000  # a 64 KB-aligned non-null address: host checks never dereference it
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3


@pytest.fixture(scope="module")
def L():
    sv.build()
    return sv.lib()


def cache(**over):
    a = dict(k=FAKE, v=FAKE, page_table=FAKE, lens=FAKE, layer_stride=0, page_stride=16 * 2 * 64,
             row_stride=128, head_stride=64, layers=1, pages=9, page_size=16, max_pages=4,
             table_stride=4, heads=2, head_dim=64, dtype=1)
    a.update(over)
    return struct.pack("@4P4q8i", *[x or 0 for x in a.values()])  # specv_cache


def rows(data=FAKE, b=64 * 32, n=64 * 8, h=64):
    return struct.pack("@P3q", data or 0, b, n, h)  # specv_rows


BAD_CACHES = [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(page_table=None), INVALID),
    (dict(lens=None), INVALID), (dict(dtype=0), INVALID), (dict(dtype=3), INVALID),
    (dict(k=FAKE + 8), INVALID), (dict(v=FAKE + 2), INVALID), (dict(page_table=FAKE + 2), INVALID),
    (dict(lens=FAKE + 1), INVALID), (dict(page_stride=2047), INVALID), (dict(row_stride=4), INVALID),
    (dict(head_stride=63), INVALID), (dict(layer_stride=1), INVALID), (dict(pages=0), INVALID),
    (dict(page_size=0), INVALID), (dict(max_pages=0), INVALID), (dict(table_stride=3), INVALID),
    (dict(heads=0), INVALID), (dict(layers=0), INVALID), (dict(head_dim=0), INVALID),
    (dict(head_dim=136), UNSUPPORTED), (dict(head_dim=60), UNSUPPORTED), (dict(heads=2000), UNSUPPORTED),
]


def append(L, c=None, **over):
    a = dict(cache=c or cache(), q=rows(), k=rows(), v=rows(), parents=FAKE, nodes=FAKE, B=2, N=4,
             heads=4, qw=FAKE, kw=FAKE, eps=1e-6, inv=FAKE, rot=64, inter=0, scale=1.0, out=rows(),
             status=FAKE)
    a.update(over)
    return L.spec_append_nodes(a["cache"], a["q"], a["k"], a["v"], a["parents"], a["nodes"], a["B"],
                               a["N"], a["heads"], a["qw"], a["kw"], a["eps"], a["inv"], a["rot"],
                               a["inter"], a["scale"], a["out"], a["status"], None)


def attend(L, c=None, **over):
    a = dict(cache=c or cache(), q=rows(), parents=FAKE, nodes=FAKE, B=2, N=4, heads=4, scale=0.1,
             out=rows(), status=FAKE, ws=FAKE, bytes=1 << 40)
    a.update(over)
    return L.spec_tree_attention(a["cache"], a["q"], a["parents"], a["nodes"], a["B"], a["N"],
                                 a["heads"], a["scale"], a["out"], a["status"], a["ws"], a["bytes"],
                                 None)


def keep(L, c=None, **over):
    a = dict(cache=c or cache(), path=FAKE, acc=FAKE, B=2, N=4, new=FAKE + 64, status=FAKE)
    a.update(over)
    return L.spec_keep_path(a["cache"], a["path"], a["acc"], a["B"], a["N"], a["new"], a["status"], None)


def process(L, **over):
    a = dict(z=FAKE, bs=400, rs=100, dtype=1, B=2, R=4, V=100, tokens=FAKE, parents=FAKE, rows=FAKE,
             hist=FAKE, hs=10, len=10, seq=FAKE, prompt=FAKE, rho=FAKE, freq=FAKE, pres=FAKE, bt=FAKE,
             bv=FAKE, nb=3, allowed=FAKE, out=FAKE, obs=400, ors=100, status=FAKE)
    a.update(over)
    return L.spec_process_logits(*a.values(), None)


@pytest.mark.parametrize("call", [append, attend, keep])
def test_cache_limits(L, call):
    for over, status in BAD_CACHES:
        assert call(L, cache(**over)) == status, over
    for over, status in [(dict(B=0), INVALID), (dict(N=0), INVALID), (dict(B=65536), UNSUPPORTED),
                         (dict(N=65), UNSUPPORTED)]:
        assert call(L, **over) == status, over
    assert call(L, cache(table_stride=0), B=2) == INVALID


@pytest.mark.parametrize("over,status", [
    (dict(q=rows(None)), 1), (dict(k=rows(FAKE + 8)), 1), (dict(v=rows(n=4)), 1), (dict(out=rows(h=63)), 1),
    (dict(q=None), 1), (dict(status=None), 1), (dict(heads=0), 1), (dict(heads=1025), 2),
    (dict(rot=63), 1), (dict(rot=66), 1), (dict(rot=-2), 1), (dict(rot=0), 1), (dict(inv=None), 1),
    (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1),
    (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(qw=FAKE + 2), 1),
    (dict(kw=FAKE + 8), 1), (dict(parents=FAKE + 2), 1), (dict(nodes=FAKE + 1), 1),
    (dict(status=FAKE + 2), 1), (dict(inv=FAKE + 2), 1),
])
def test_append_refusals(L, over, status):
    assert append(L, **over) == status
    assert append(L, cache(layers=2)) == INVALID


@pytest.mark.parametrize("over,status", [
    (dict(q=rows(None)), 1), (dict(out=rows(FAKE + 4)), 1), (dict(out=None), 1), (dict(q=rows(b=12)), 1),
    (dict(status=None), 1), (dict(ws=None), 1), (dict(ws=FAKE + 128), 1), (dict(bytes=16), 3),
    (dict(heads=3), 1), (dict(heads=0), 1), (dict(heads=1026), 2), (dict(scale=0.0), 1),
    (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1),
    (dict(parents=FAKE + 1), 1), (dict(nodes=FAKE + 2), 1), (dict(status=FAKE + 1), 1),
])
def test_attention_refusals(L, over, status):
    assert attend(L, **over) == status
    assert attend(L, cache(layers=2)) == INVALID


@pytest.mark.parametrize("over,status", [
    (dict(path=None), 1), (dict(acc=None), 1), (dict(new=None), 1), (dict(status=None), 1),
    (dict(new=FAKE), 1), (dict(path=FAKE + 2), 1), (dict(acc=FAKE + 1), 1), (dict(new=FAKE + 66), 1),
    (dict(status=FAKE + 2), 1),
])
def test_keep_refusals(L, over, status):
    assert keep(L, **over) == status
    assert keep(L, cache(layers=70000)) == UNSUPPORTED


@pytest.mark.parametrize("over,status", [
    (dict(z=None), 1), (dict(out=None), 1), (dict(hist=None), 1), (dict(seq=None), 1),
    (dict(status=None), 1), (dict(tokens=None), 1), (dict(dtype=2), 1), (dict(B=0), 1), (dict(R=0), 1),
    (dict(V=0), 1), (dict(len=-1), 1), (dict(nb=-1), 1), (dict(bt=None), 1), (dict(bv=None), 1),
    (dict(z=FAKE + 1), 1), (dict(out=FAKE + 1), 1), (dict(hist=FAKE + 2), 1), (dict(allowed=FAKE + 2), 1),
    (dict(rho=FAKE + 2), 1), (dict(ors=101), 1), (dict(obs=800), 1), (dict(R=65), 2), (dict(B=65536), 2),
    (dict(V=1048577), 2), (dict(dtype=0, V=524289), 2), (dict(nb=1025), 2), (dict(len=2 ** 28 + 1), 2),
])
def test_process_refusals(L, over, status):
    assert process(L, **over) == status


@pytest.mark.parametrize("over", [dict(b=-64 * 32), dict(n=-64 * 8), dict(h=-64)])
def test_strides_below_zero_are_refused(L, over):
    for name in ("q", "k", "v", "out"):
        assert append(L, **{name: rows(**over)}) == INVALID
    for name in ("q", "out"):
        assert attend(L, **{name: rows(**over)}) == INVALID
    for call in (append, attend, keep):
        assert call(L, cache(page_stride=-16 * 2 * 64)) == INVALID
        assert call(L, cache(row_stride=-128)) == INVALID
        assert call(L, cache(head_stride=-64)) == INVALID
        assert call(L, cache(layer_stride=-8)) == INVALID
    for name in ("bs", "rs", "obs", "ors", "hs"):
        assert process(L, **{name: -1000}) == INVALID


FAKE_ATTRIBUTE = r"""
#include <stdio.h>
int cudaFuncSetAttribute(const void* f, int attribute, int value) {
  fprintf(stderr, "limit %p %d %d\n", f, attribute, value);
  return 1;  // refused: the call ends here, before any launch
}
"""

CALLS = """
import sys
sys.path[:0] = {paths!r}
import speculative_decoding_verify_sample_gb300 as sv, test_tree_cpu as t
L = sv.lib()
for dtype in (0, 1):
    for B, R, V in ((10, 2, 65536), (60, 4, 65536), (8, 33, 100000)):
        for length, biases in ((1, 0), (300, 7), (9000, 1024)):
            assert t.process(L, dtype=dtype, B=B, R=R, V=V, len=length, hs=length, nb=biases,
                             bs=R * V, obs=R * V, rs=V, ors=V) == 4  # SPECV_ERR_CUDA
"""


def test_logits_shared_memory_limit_is_the_same_for_every_call(L, tmp_path):
    """The limit belongs to the kernel, not to a call: if calls set limits of their own, one in
    another thread could lower it between this call's setting and its launch."""
    fake, lib = tmp_path / "fake.c", str(tmp_path / "fake.so")
    fake.write_text(FAKE_ATTRIBUTE)
    subprocess.run(["gcc", "-shared", "-fPIC", str(fake), "-o", lib], check=True)
    here = os.path.dirname(os.path.abspath(__file__))
    run = subprocess.run([sys.executable, "-c", CALLS.format(paths=[here, os.path.dirname(here)])],
                         env=dict(os.environ, LD_PRELOAD=lib), capture_output=True, text=True)
    assert run.returncode == 0, run.stderr
    limits = {}
    for line in run.stderr.splitlines():
        if line.startswith("limit "):
            _, kernel, attribute, value = line.split()
            limits.setdefault((kernel, attribute), []).append(int(value))
    assert len(limits) == 4 and all(len(v) >= 3 for v in limits.values())  # two sizes, two types
    assert all(len(set(v)) == 1 for v in limits.values()), limits


def test_attention_workspace_sizes(L):
    size = L.specv_attention_workspace_bytes
    assert size(1, 1, 1, 1, 8) > 0
    assert size(256, 64, 64, 8, 128) >= size(1, 64, 64, 8, 128)
    for bad in [(0, 1, 1, 1, 64), (1, 0, 1, 1, 64), (1, 65, 1, 1, 64), (1, 1, 3, 2, 64), (1, 1, 0, 1, 64),
                (1, 1, 1, 0, 64), (1, 1, 1, 1, 136), (1, 1, 1, 1, 12), (1, 1, 2048, 1, 64), (65536, 1, 1, 1, 64)]:
        assert size(*bad) == 0, bad
    with pytest.raises(ValueError):
        sv.AttentionWorkspace(1, 65, 8, 8, 128)


def test_struct_layouts_match_the_header(tmp_path):
    """The packed bytes are the header's structs: sizes and offsets by the C compiler."""
    probe = tmp_path / "probe.c"
    probe.write_text('#include <stdio.h>\n#include "specverify.h"\n'
                     'int main(void) { printf("%zu %zu %zu %zu %zu", sizeof(specv_cache), '
                     'offsetof(specv_cache, layer_stride), offsetof(specv_cache, layers), '
                     'offsetof(specv_cache, dtype), sizeof(specv_rows)); return 0; }')
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    exe = str(tmp_path / "probe")
    subprocess.run(["gcc", "-I", os.path.join(root, "include"), str(probe), "-o", exe], check=True)
    said = [int(x) for x in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    assert said == [struct.calcsize("@4P4q8i"), struct.calcsize("@4P"), struct.calcsize("@4P4q"),
                    struct.calcsize("@4P4q7i"), struct.calcsize("@P3q")]


def _tensors(B=2, N=3, Hq=4, Hkv=2, D=64, page=16, P=3, dtype=torch.bfloat16):
    return dict(q=torch.zeros(B, N, Hq, D, dtype=dtype), kv=torch.zeros(B, N, Hkv, D, dtype=dtype),
                cache=torch.zeros(B * P, page, Hkv, D, dtype=dtype),
                table=torch.zeros(B, P, dtype=torch.int32), lens=torch.zeros(B, dtype=torch.int32))


def test_binding_refuses_wrong_tensors():
    t = _tensors()
    q, kv, c, table, lens = t["q"], t["kv"], t["cache"], t["table"], t["lens"]
    with pytest.raises(ValueError, match="CUDA"):
        sv.tree_attention(q, c, c, table, lens)
    with pytest.raises(ValueError, match="CUDA"):
        sv.append_nodes(q, kv, kv, c, c, table, lens)
    with pytest.raises(ValueError, match="CUDA"):
        sv.keep_path(lens[:, None], lens, c, c, table, lens)
    with pytest.raises(ValueError, match="CUDA"):
        sv.process_logits(torch.zeros(2, 9), table, lens)
    for bad in [dict(c=c.float()), dict(c=c[0])]:
        with pytest.raises((TypeError, ValueError)):
            sv.tree_attention(q, bad["c"], bad["c"], table, lens)
    with pytest.raises(ValueError):
        sv.tree_attention(q, c, c[:, :8], table, lens)              # another shape
    with pytest.raises(ValueError):
        sv.tree_attention(q, c, c.transpose(1, 2).contiguous().transpose(1, 2), table, lens)  # strides
    with pytest.raises(ValueError):
        sv.tree_attention(q.half(), c, c, table, lens)
    with pytest.raises(ValueError):
        sv.tree_attention(q[:, :, :3], c, c, table, lens)           # heads that do not divide
    with pytest.raises(ValueError):
        sv.tree_attention(q, c, c, table.long(), lens)
    with pytest.raises(ValueError):
        sv.tree_attention(q, c, c, table, lens[:1])
    with pytest.raises(ValueError):
        sv.tree_attention(q, c, c, table, lens, torch.zeros(2, 4, dtype=torch.int32))
    with pytest.raises(ValueError):
        sv.tree_attention(q, c, c, table, lens, None, lens.long())
    with pytest.raises(ValueError):
        sv.tree_attention(q[0], c, c, table, lens)
    with pytest.raises(ValueError):
        sv.append_nodes(q, kv[:, :, :1], kv, c, c, table, lens)
    with pytest.raises(ValueError):
        sv.append_nodes(q, kv, kv, c, c, table, lens, torch.zeros(8, dtype=torch.float64))
    with pytest.raises(ValueError):
        sv.append_nodes(q, kv, kv, c, c, table, lens, q_weight=torch.ones(64))
    with pytest.raises(ValueError):
        sv.keep_path(lens, lens, c, c, table, lens)
    z, hist = torch.zeros(2, 3, 9), torch.zeros(2, 5, dtype=torch.int32)
    with pytest.raises(ValueError):
        sv.process_logits(z, hist, lens)                            # rows without tokens
    with pytest.raises(ValueError):
        sv.process_logits(z, hist, lens, tokens=torch.zeros(2, 3, dtype=torch.int32))
    with pytest.raises(ValueError):
        sv.process_logits(z[:, 0], hist, lens, bias_tokens=hist)
    with pytest.raises(ValueError):
        sv.process_logits(z[:, 0], hist, lens, allowed=torch.zeros(2, 2, dtype=torch.int32))
    with pytest.raises(TypeError):
        sv.process_logits(z[:, 0].half(), hist, lens)
    with pytest.raises(ValueError):
        sv.process_logits(z[:, 0], hist.float(), lens)


def test_star_import_needs_no_torch():
    """Everything the package names can be imported where torch cannot."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([sys.executable, "-c", "import sys; sys.modules['torch'] = None\n"
                    "from speculative_decoding_verify_sample_gb300 import *\n"
                    "import speculative_decoding_verify_sample_gb300 as sv\n"
                    "assert all(callable(globals()[n]) or n.startswith('DEV_') for n in sv.__all__)\n"
                    "assert tree_attention is sv.tree_attention"], cwd=root, check=True)


@pytest.mark.parametrize("why", ["no compiler", "failed", "no CUDA"])
def test_build_without_the_extension_leaves_the_library(monkeypatch, tmp_path, why):
    """build() warns and returns, a stale extension is gone, and a call that needs it says why."""
    import importlib

    how = importlib.import_module("speculative_decoding_verify_sample_gb300.build")
    tree = importlib.import_module("speculative_decoding_verify_sample_gb300.tree")
    built, path = [], tmp_path / "extension.so"
    path.write_text("of an older source")
    os.utime(path, (1, 1))
    for module in (how, tree):
        monkeypatch.setattr(module, "binding_path", lambda: str(path))
    monkeypatch.setattr(how, "_build_library", lambda *a: built.append(a))
    monkeypatch.setattr(how, "_binding_failure", None)
    monkeypatch.setattr(tree, "_binding", None)
    if why == "no CUDA":
        monkeypatch.setattr(torch.version, "cuda", None)
    else:
        monkeypatch.setenv("CXX", str(tmp_path / "none") if why == "no compiler" else "false")
    with pytest.warns(UserWarning, match="without the drafted tree's operators"):
        assert how.build() == how.LIB_PATH
    assert built and not path.exists()
    reason = {"no compiler": "No such file", "failed": "false failed", "no CUDA": "no CUDA"}[why]
    t = _tensors()
    with pytest.raises(RuntimeError, match=reason):
        sv.tree_attention(t["q"], t["cache"], t["cache"], t["table"], t["lens"])


def test_binding_refuses_a_stream_of_another_device(monkeypatch):
    """The extension answers None where the tensors are not on the current device: with such a
    stream it does so twice."""
    import contextlib
    import types

    tree = sv.tree
    monkeypatch.setattr(tree, "_there", lambda device, stream: contextlib.nullcontext())
    tensor = types.SimpleNamespace(is_cuda=True, device="cuda:1")
    with pytest.raises(ValueError, match="stream is of another device than the tensors, on cuda:1"):
        tree._call("spec_keep_path", lambda: None, tensor, object())
    answers = iter([None, ("out", "status")])  # tensors of another device than the current one
    assert tree._call("spec_keep_path", lambda: next(answers), tensor, None) == ("out", "status")


def test_binding_refuses_sizes_past_32_bits():
    """Each with a ValueError that names it: not behind the point where Python's lock is given up."""
    big = 2 ** 31 + 7

    def t(*shape, dtype=torch.int32):
        return torch.empty(shape, dtype=dtype, device="meta")  # takes no memory

    bf16, c = torch.bfloat16, t(9, 16, 1, 8, dtype=torch.bfloat16)
    one = t(1, 1, 1, 8, dtype=bf16)
    for name, call in [
        ("V", lambda: sv.process_logits(t(1, big, dtype=bf16), t(1, 5), t(1))),
        ("L", lambda: sv.process_logits(t(1, 9, dtype=bf16), t(1, big), t(1))),
        ("B", lambda: sv.process_logits(t(big, 9, dtype=bf16), t(big, 5), t(big))),
        ("R", lambda: sv.process_logits(t(1, big, 9, dtype=bf16), t(1, 5), t(1), tokens=t(1, big - 1))),
        ("biases", lambda: sv.process_logits(t(1, 9, dtype=bf16), t(1, 5), t(1), bias_tokens=t(1, big),
                                             bias_values=t(1, big, dtype=torch.float32))),
        ("B", lambda: sv.tree_attention(t(big, 1, 1, 8, dtype=bf16), c, c, t(big, 3), t(big))),
        ("N", lambda: sv.tree_attention(t(1, big, 1, 8, dtype=bf16), c, c, t(1, 3), t(1))),
        ("q_heads", lambda: sv.tree_attention(t(1, 1, big, 8, dtype=bf16), c, c, t(1, 3), t(1))),
        ("q_heads", lambda: sv.append_nodes(t(1, 1, big, 8, dtype=bf16), one, one, c, c, t(1, 3), t(1))),
        ("inv_freq", lambda: sv.append_nodes(one, one, one, c, c, t(1, 3), t(1),
                                             t(2 ** 30, dtype=torch.float32))),
        ("B", lambda: sv.keep_path(t(big, 2), t(big), c, c, t(big, 3), t(big))),
        ("N", lambda: sv.keep_path(t(1, big), t(1), c, c, t(1, 3), t(1))),
    ]:
        with pytest.raises(ValueError, match=f"^{name} is too large"):
            call()


# ---------------------------------------------------- the plain forms themselves


def test_plain_attention_of_a_chain_is_causal_attention():
    k, v, table = ref.make_cache(1, 1, 4, 1, 8, 4, [6], torch.float32, "cpu", fill=0.0)
    k, v = torch.randn_like(k), torch.randn_like(v)
    q = torch.randn(1, 4, 2, 8)
    out, *_ = ref.attention(q, k, v, table, [6], None, [4], 0.3)
    pg, off = ref.slots(table, 0, 4, list(range(10)), "cpu")
    kk, vv = k[pg, off, 0].double(), v[pg, off, 0].double()
    s = torch.einsum("ihd,jd->hij", q[0].double(), kk) * 0.3
    s = s.masked_fill(torch.ones(4, 10, dtype=torch.bool).triu(7), float("-inf"))
    want = torch.einsum("hij,jd->ihd", s.softmax(-1), vv)
    assert (out[0] - want).abs().max() < 1e-12


def test_plain_rotation_keeps_lengths_and_relative_angles():
    inv = torch.tensor([1.0, 0.1, 0.01])
    x, y = torch.randn(1, 8), torch.randn(1, 8)
    for inter in (False, True):
        dots = []
        for shift in (0, 1000):
            a, _ = ref.append(x, torch.tensor(3 + shift), None, 0, inv, inter, 1.0)
            b, _ = ref.append(y, torch.tensor(10 + shift), None, 0, inv, inter, 1.0)
            dots.append((a * b).sum().item())
            assert abs(a.norm() - x.double().norm()) < 1e-9
        assert abs(dots[0] - dots[1]) < 1e-4  # inv_freq is in 32 bits


def test_plain_logits_by_hand():
    z = np.array([[[1.0, -1.0, 2.0, 0.5]]] * 2)
    out, _ = ref.logits(z, np.array([[0, 1, 1], [2, 2, 2]]), [3, 1], [1, 1], np.zeros((2, 0), int), None,
                        [1, 1], [2.0, 4.0], [0.25, 0.25], [0.5, 0.5], np.array([[3, 3], [3, -1]]),
                        np.array([[1.0, 1.0], [1.0, 1.0]]), np.array([[[0b1011]], [[0b1111]]], np.int32))
    assert out[0, 0].tolist() == [0.5, -3.0, -np.inf, 2.5]
    assert out[1, 0].tolist() == [1.0, -1.0, 0.5, 1.5]
