"""The operators on a drafted tree against plain 64-bit forms: the append of
the nodes' projections, the attention over the paged cache, the penalties and
masks on the logits, the move of the accepted path's rows, and all of them
together as a serving step runs them."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import tree_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verify_sample_gb300 as sv
    sv.build()
    sv.lib()
    return sv


def i32(a):
    return torch.as_tensor(np.ascontiguousarray(a, np.int32)).cuda()


def f32(a):
    return torch.as_tensor(np.ascontiguousarray(a, np.float32)).cuda()


def close(got, want, tol, label=""):
    """Element by element; NaN and infinities where the reference has them."""
    got, want, tol = (torch.as_tensor(x).double().cpu() for x in (got, want, tol))
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), label
    odd = ~fine & ~torch.isnan(want)
    assert torch.equal(got[odd], want[odd]), label
    off = (got - want).abs()[fine]
    worst = (off / tol[fine]).max().item() if off.numel() else 0.0
    assert worst <= 1.0, (label, worst, off.max().item())


# ------------------------------------------------------------------ attention


class Attn:
    """One call's inputs and its reference."""

    def __init__(self, seed, B, N, Hq, Hkv, D, page, lens, dtype, *, chain=False, nodes=None,
                 layout="rows", scale=None, sharp=1.0):
        rng = np.random.default_rng(seed)
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.B, self.N, self.Hq, self.D, self.dtype = B, N, Hq, D, dtype
        self.lens = [int(x) for x in lens]
        self.k, self.v, self.table = ref.make_cache(seed, B, N, Hkv, D, page, self.lens, dtype, "cuda",
                                                    layout=layout)
        self.page = page
        self.parents = None if chain else ref.random_parents(rng, B, N)
        self.nodes = np.full(B, N) if nodes is None else np.asarray(nodes)
        for b in range(B):
            at = range(self.lens[b], self.lens[b] + int(self.nodes[b]))
            pg, off = ref.slots(self.table, b, page, list(at), "cuda")
            for c in (self.k, self.v):
                c[pg, off] = torch.randn(len(at), Hkv, D, generator=gen, device="cuda").to(dtype)
        self.q = (sharp * torch.randn(B, N, Hq, D, generator=gen, device="cuda")).to(dtype)
        self.scale = scale
        self.given_nodes = nodes is not None

    def args(self):
        return (self.q, self.k, self.v, self.table, i32(self.lens),
                None if self.parents is None else i32(self.parents),
                i32(self.nodes) if self.given_nodes else None)

    def want(self, many=False):
        scale = self.scale if self.scale is not None else self.D ** -0.5
        parts = (ref.attention_of_many if many else ref.attention)(
            self.q, self.k, self.v, self.table, self.lens, self.parents, self.nodes, scale)
        keys = max(self.lens) + self.N
        return parts, ref.attention_tolerance(parts, self.D, keys, self.dtype)

    def check(self, sv, **kw):
        out = torch.full(self.q.shape, 7.0, dtype=self.dtype, device="cuda")
        if self.scale is not None:
            kw["scale"] = self.scale
        got, status = sv.tree_attention(*self.args(), out=out, **kw)
        torch.cuda.synchronize()
        assert got is out
        assert status.tolist() == [0] * self.B
        (want, *_), tol = self.want()
        for b in range(self.B):
            n = int(self.nodes[b])
            close(got[b, :n], want[b, :n], tol[b, :n], f"request {b}")
            assert (got[b, n:] == 7.0).all()  # rows behind the last node


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("B,N,Hq,Hkv,D,page,lens,chain,nodes", [
    (1, 1, 1, 1, 8, 16, [0], True, None),                # the root alone: no cache
    (1, 1, 8, 8, 64, 16, [1], True, None),
    (2, 1, 8, 1, 128, 16, [127, 128], True, None),       # plain decoding at a tile's edge
    (3, 1, 12, 4, 128, 64, [0, 1, 129], True, None),
    (1, 5, 32, 8, 128, 16, [300], True, None),           # K = 4 drafts
    (2, 64, 8, 1, 64, 32, [65, 191], True, None),        # the longest chain, 512 rows
    (2, 64, 6, 2, 128, 128, [0, 100], False, None),
    (3, 32, 16, 2, 128, 64, [31, 257, 1000], False, [32, 1, 17]),
    (2, 7, 7, 1, 80, 24, [50, 333], False, None),        # heads that are no power of two
    (2, 9, 9, 3, 96, 1, [5, 140], False, [9, 3]),        # a page to each token
    (1, 33, 4, 4, 120, 100, [513], False, None),
    (2, 3, 10, 2, 24, 3, [77, 0], False, [2, 3]),
    (1, 16, 64, 4, 112, 200, [900], False, None),
    (4, 2, 2, 2, 40, 8, [3, 0, 254, 126], False, [1, 2, 2, 1]),
])
def test_attention(sv, dtype, B, N, Hq, Hkv, D, page, lens, chain, nodes):
    Attn(11 * N + B, B, N, Hq, Hkv, D, page, lens, dtype, chain=chain, nodes=nodes).check(sv)


@pytest.mark.parametrize("layout", ["heads", "pairs"])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_attention_cache_layouts(sv, layout, dtype):
    Attn(5, 2, 6, 8, 2, 64, 16, [200, 37], dtype, layout=layout).check(sv)


@pytest.mark.parametrize("page", [2, 4, 8, 12, 40, 48, 96, 136, 192, 384, 1000])
@pytest.mark.parametrize("layout", ["rows", "heads"])
def test_attention_page_sizes(sv, page, layout):
    """Pages that tiles are made of, or that end inside one."""
    Attn(page, 3, 5, 8, 2, 128, page, [700, 127, 2 * page + 1], BF16, layout=layout).check(sv)


@pytest.mark.parametrize("lens,N", [([5000], 1), ([4097, 3, 2999], 4), ([2500, 2501], 40)])
def test_attention_long_contexts(sv, lens, N):
    """Enough keys that a request's are shared out over the machine."""
    Attn(3, len(lens), N, 8, 2, 128, 64, lens, BF16, chain=N == 4).check(sv)


def test_attention_many_short_requests(sv):
    lens = np.random.default_rng(2).integers(0, 90, 300)
    nodes = np.random.default_rng(4).integers(1, 4, 300)
    Attn(8, 300, 3, 4, 2, 64, 16, lens, BF16, nodes=nodes).check(sv)


@pytest.mark.parametrize("dtype,B,N,Hq,Hkv,D,page,most", [
    (BF16, 24, 4, 32, 8, 128, 16, 3000),     # at most 64 rows
    (F16, 40, 13, 32, 8, 64, 64, 2000),
    (BF16, 24, 32, 32, 8, 128, 64, 2900),    # at most 128
    (F16, 30, 16, 16, 2, 80, 128, 9000),
    (BF16, 20, 20, 24, 6, 128, 24, 2900),    # pages that end inside a tile
    (BF16, 16, 64, 32, 4, 128, 256, 4500),   # more: two row tiles on the same keys, two of them
    (F16, 20, 40, 40, 8, 64, 32, 2300),
    (BF16, 16, 33, 48, 6, 112, 100, 3000),
])
def test_attention_fills_the_machine(sv, dtype, B, N, Hq, Hkv, D, page, most):
    """More work than eight tiles for each SM: items cut anywhere, trees that lie
    across tiles; the same bits every time."""
    rng = np.random.default_rng(B)
    lens = rng.integers(0, most, B)
    lens[:4] = [most, 870, 127, 128 * 7 - 1]
    a = Attn(B + N, B, N, Hq, Hkv, D, page, lens, dtype, nodes=rng.integers(1, N + 1, B))
    tiles = sum(-(-(x + N) // 128) for x in a.lens) * Hkv * -(-N * Hq // Hkv // 256)
    assert tiles > 8 * 152
    parts, tol = a.want(many=True)
    args, ws = a.args(), sv.AttentionWorkspace(B, N, Hq, Hkv, D, device="cuda")
    first = None
    for _ in range(4):
        out = torch.full(a.q.shape, 7.0, dtype=dtype, device="cuda")
        got, status = sv.tree_attention(*args, out=out, workspace=ws)
        assert status.tolist() == [0] * B
        for b in range(B):
            n = int(a.nodes[b])
            close(got[b, :n], parts[0][b, :n], tol[b, :n], f"request {b}")
            assert (got[b, n:] == 7.0).all()
        assert first is None or torch.equal(got, first)
        first = got.clone()


@pytest.mark.parametrize("sharp", [0.0, 12.0])
def test_attention_flat_and_sharp_scores(sv, sharp):
    """All scores equal; scores far apart, whose running maximum moves much."""
    Attn(6, 2, 8, 8, 2, 128, 32, [700, 1300], BF16, sharp=sharp).check(sv)


def test_attention_scale_and_rising_maxima(sv):
    """The largest score last: every tile raises the maximum by much."""
    a = Attn(9, 1, 4, 4, 1, 64, 32, [1500], F16, chain=True, scale=0.5)
    pg, off = ref.slots(a.table, 0, 32, list(range(1504)), "cuda")
    ramp = torch.linspace(-40, 40, 1504, device="cuda")[:, None, None]
    a.k[pg, off] = (ramp * torch.ones(1504, 1, 64, device="cuda") / 8).to(F16)
    a.q[:] = 0.25
    a.check(sv)


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("where", ["k", "v"])
@pytest.mark.parametrize("N,Hq", [(8, 8), (64, 16)])
def test_attention_masked_places_hold_anything(sv, bad, where, N, Hq):
    """A node's key or value is NaN or infinite: only it and its descendants see it."""
    a = Attn(21, 1, N, Hq, 2, 64, 16, [120], BF16)
    pg, off = ref.slots(a.table, 0, 16, [120 + 2], "cuda")
    cache = getattr(a, where)
    cache[pg, off, :, 5] = bad
    out, _ = sv.tree_attention(*a.args())
    (want, *_), tol = a.want()
    hit = [i for i in range(N) if 2 in ref.path_of(a.parents, 0, i)]
    clean = [i for i in range(N) if i not in hit]
    assert hit and clean
    close(out[0, clean], want[0, clean], tol[0, clean])
    if where == "v":
        others = [d for d in range(64) if d != 5]
        close(out[0, hit][..., others], want[0, hit][..., others], tol[0, hit][..., others])
        got, expected = out[0, hit][..., 5].double(), want[0, hit][..., 5]
        assert torch.equal(torch.isnan(got), torch.isnan(expected))
        assert torch.equal(torch.isinf(got), torch.isinf(expected))
    else:  # a score of -inf (an infinite key against a negative query) takes its key out
        assert torch.equal(torch.isnan(out[0, hit].double()), torch.isnan(want[0, hit]))


def test_attention_lowest_values_in_the_cache(sv):
    """Keys at the type's lowest values: scores of -inf beside finite ones."""
    a = Attn(22, 1, 2, 2, 1, 64, 16, [140], BF16, chain=True)
    pg, off = ref.slots(a.table, 0, 16, list(range(0, 140, 3)), "cuda")
    a.k[pg, off] = torch.finfo(BF16).min
    a.q.abs_()
    out, _ = sv.tree_attention(*a.args())
    keep = [s for s in range(142) if s >= 140 or s % 3]
    b = Attn(22, 1, 2, 2, 1, 64, 16, [140], BF16, chain=True)
    b.q.abs_()
    for i in range(2):
        seen = [s for s in keep if s <= 140 + i]
        pg, off = ref.slots(b.table, 0, 16, seen, "cuda")
        s = torch.einsum("hd,jhd->hj", b.q[0, i].double(), b.k[pg, off].double().expand(-1, 2, -1)) / 8
        want = torch.einsum("hj,jhd->hd", s.softmax(-1), b.v[pg, off].double().expand(-1, 2, -1))
        mass = torch.einsum("hj,jhd->hd", s.softmax(-1), b.v[pg, off].double().abs().expand(-1, 2, -1))
        close(out[0, i], want, mass * (2.0 ** -8 + 2.0 ** -12) + want.abs() * 2.0 ** -8 * 1.01)


def test_attention_strided_queries_and_outputs(sv):
    a = Attn(13, 2, 5, 8, 2, 64, 16, [90, 33], BF16)
    qkv = torch.randn(2, 5, 12 * 64, device="cuda").to(BF16)
    qkv[..., :512] = a.q.flatten(2)
    a.q = qkv[..., :512].unflatten(-1, (8, 64))
    wide = torch.full((2, 5, 8, 128), 7.0, dtype=BF16, device="cuda")
    got, _ = sv.tree_attention(*a.args(), out=wide[..., 64:])
    (want, *_), tol = a.want()
    close(got, want, tol)
    assert (wide[..., :64] == 7.0).all()


def test_attention_offsets_past_32_bits(sv):
    """Pages more than 2^31 elements into the cache."""
    page, Hkv, D = 16, 2, 128
    far = (2 ** 31 + 2 ** 27) // (page * Hkv * D)
    k = torch.zeros(far, page, Hkv, D, dtype=BF16, device="cuda")
    v = torch.zeros_like(k)
    table = i32([[far - 1, 3, far - 7]])
    for pg in (far - 1, 3, far - 7):
        k[pg] = torch.randn(page, Hkv, D, device="cuda").to(BF16)
        v[pg] = torch.randn(page, Hkv, D, device="cuda").to(BF16)
    q = torch.randn(1, 3, 4, D, device="cuda").to(BF16)
    out, status = sv.tree_attention(q, k, v, table, i32([44]))
    parts = ref.attention(q, k, v, table, [44], None, [3], D ** -0.5)
    close(out, parts[0], ref.attention_tolerance(parts, D, 48, BF16))
    assert status.tolist() == [0]


def _bad_requests(sv, call, good):
    """call(n_nodes, lens, parents, table) -> (rows [B, ...], status); each kind
    of bad data flags its request, zeroes its rows and leaves the others alone."""
    B, N = 5, 4
    parents = np.array([[-1, 0, 0, 2]] * B)
    nodes, lens, table = np.full(B, N), np.array([30, 31, 32, 33, 34]), good.copy()
    clean, status = call(nodes, lens, parents, table)
    assert status.tolist() == [0] * B
    for change, bit in [
        (lambda n, l, p, t: n.__setitem__(1, 0), sv.DEV_BAD_DRAFT_LEN),
        (lambda n, l, p, t: n.__setitem__(1, N + 1), sv.DEV_BAD_DRAFT_LEN),
        (lambda n, l, p, t: l.__setitem__(1, -1), sv.DEV_BAD_CACHE),
        (lambda n, l, p, t: l.__setitem__(1, 8 * t.shape[1] - 3), sv.DEV_BAD_CACHE),
        (lambda n, l, p, t: l.__setitem__(1, 2 ** 31 - 1), sv.DEV_BAD_CACHE),
        (lambda n, l, p, t: p.__setitem__((1, 2), 2), sv.DEV_BAD_TREE),
        (lambda n, l, p, t: p.__setitem__((1, 0), 0), sv.DEV_BAD_TREE),
        (lambda n, l, p, t: p.__setitem__((1, 3), -1), sv.DEV_BAD_TREE),
        (lambda n, l, p, t: t.__setitem__((1, 4), 10 ** 6), sv.DEV_BAD_CACHE),
        (lambda n, l, p, t: t.__setitem__((1, 4), -1), sv.DEV_BAD_CACHE),
    ]:
        data = [x.copy() for x in (nodes, lens, parents, table)]
        change(*data)
        rows, status = call(*data)
        assert status.tolist() == [0, bit, 0, 0, 0], (bit, status.tolist())
        for b in (0, 2, 3, 4):
            assert torch.equal(rows[b], clean[b])
        assert (rows[1] == 0).all()


def test_attention_flags_bad_requests(sv):
    a = Attn(31, 5, 4, 4, 2, 64, 8, [30, 31, 32, 33, 34], BF16)

    def call(nodes, lens, parents, table):
        out = torch.full(a.q.shape, 7.0, dtype=BF16, device="cuda")
        return sv.tree_attention(a.q, a.k, a.v, i32(table), i32(lens), i32(parents), i32(nodes),
                                 out=out)

    _bad_requests(sv, call, a.table.cpu().numpy())


@pytest.mark.parametrize("page,N,Hq", [(32, 4, 4), (64, 4, 4), (128, 4, 4), (16, 64, 8), (32, 64, 8),
                                       (128, 64, 8)])
@pytest.mark.parametrize("bad_page", [-1, 10 ** 6, 2 ** 31 - 1])
def test_attention_flags_bad_pages_of_tensor_copies(sv, page, N, Hq, bad_page):
    """Pages out of range where tensor copies bring them (with more than 128 rows to a key head
    from 16 on), at a request's nodes and before them.  Nothing is copied there and nothing may be
    read, whatever the tiles held before: every place that is not a key's is NaN."""
    B, Hkv = 6, 2
    lens = [5 * page + 3, 4 * page - 2, 3 * page, 4 * page - 1, 700, 2 * page + 1]
    a = Attn(page + N, B, N, Hq, Hkv, 64, page, lens, BF16)
    q, k, v, _, lens_t, parents, _ = a.args()
    table = a.table.cpu().numpy()

    def call(pages):
        out = torch.full(q.shape, 7.0, dtype=BF16, device="cuda")
        return sv.tree_attention(q, k, v, i32(pages), lens_t, parents, out=out)

    clean, status = call(table)
    assert status.tolist() == [0] * B
    (want, *_), tol = a.want()
    close(clean, want, tol)
    for at in (0, lens[1] // page, (lens[1] + N - 1) // page):  # the first page, the nodes' first and last
        pages = table.copy()
        pages[1, at] = bad_page
        rows, status = call(pages)
        assert status.tolist() == [0, sv.DEV_BAD_CACHE] + [0] * (B - 2)
        assert (rows[1] == 0).all()
        for b in (0, 2, 3, 4, 5):
            assert torch.equal(rows[b], clean[b])


WAITS = (0, 2000, 6000, 12000, 25000)  # ns


@pytest.fixture(scope="module")
def impatient(sv, tmp_path_factory):
    """The attention with waits so short that they run out, by their length: functions like
    tree_attention of a case and an output, that return the status."""
    import ctypes
    import importlib
    import struct
    import subprocess

    from speculative_decoding_verify_sample_gb300 import _native

    how = importlib.import_module("speculative_decoding_verify_sample_gb300.build")
    where = tmp_path_factory.mktemp("impatient")
    source = next(x for x in how.SOURCES if x.endswith("attention.cu"))
    builds = [subprocess.Popen([how.nvcc_path(), *how.ARCH_FLAGS, "-O3", "-std=c++17", "-I", how.INCLUDE,
                                "-shared", "-Xcompiler", "-fPIC", "-cudart", "shared",
                                f"-DSPECV_ATTENTION_WAIT_NS={ns}ull", "-o", str(where / f"{ns}.so"), source])
              for ns in WAITS]
    assert [b.wait() for b in builds] == [0] * len(WAITS)

    def bind(ns):
        fn = ctypes.CDLL(str(where / f"{ns}.so")).spec_tree_attention
        fn.restype, fn.argtypes = _native.SIGNATURES["spec_tree_attention"]

        def call(a, args, out, ws):
            q, k, v, table, lens, parents, nodes = args
            status = i32([-1] * a.B)  # whatever was there
            cache = struct.pack("@4P4q8i", k.data_ptr(), v.data_ptr(), table.data_ptr(), lens.data_ptr(), 0,
                                *k.stride()[:3], 1, k.shape[0], k.shape[1], table.shape[1], table.stride(0),
                                k.shape[2], a.D, 1 if a.dtype == BF16 else 2)
            rows = [struct.pack("@P3q", t.data_ptr(), *t.stride()[:3]) for t in (q, out)]
            ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
            assert fn(cache, rows[0], ptr(parents), ptr(nodes), a.B, a.N, a.Hq, a.D ** -0.5, rows[1],
                      status.data_ptr(), ws.tensor.data_ptr(), ws.nbytes,
                      torch.cuda.current_stream().cuda_stream) == 0
            torch.cuda.synchronize()
            return status.tolist()

        return call

    return {ns: bind(ns) for ns in WAITS}


GIVE_UP = [  # B, N, Hq, Hkv, D, page, lens
    (3, 5, 8, 2, 128, 64, [3000, 12, 700]),           # tensor copies
    (3, 5, 8, 2, 128, 8, [3000, 12, 700]),            # copies of 16 bytes
    (2, 64, 16, 2, 128, 64, [2000, 900]),             # two row tiles
    (2, 64, 16, 2, 64, 12, [2000, 900]),
    (40, 3, 8, 2, 64, 32, [100 * (i % 7) for i in range(40)]),  # many items to a run
]


@pytest.mark.parametrize("B,N,Hq,Hkv,D,page,lens", GIVE_UP)
def test_attention_gives_up_and_leaves_the_device_usable(sv, impatient, B, N, Hq, Hkv, D, page, lens):
    """Wherever its waits run out the call ends, and those behind it are right."""
    a = Attn(71, B, N, Hq, Hkv, D, page, lens, BF16)
    args, ws = a.args(), sv.AttentionWorkspace(B, N, Hq, Hkv, D, device="cuda")
    want, _ = sv.tree_attention(*args)
    for ns in WAITS:
        for _ in range(3):
            impatient[ns](a, args, torch.zeros_like(a.q), ws)
            got, status = sv.tree_attention(*args, workspace=ws)
            assert torch.equal(got, want) and status.tolist() == [0] * B


@pytest.mark.parametrize("B,N,Hq,Hkv,D,page,lens", GIVE_UP)
def test_attention_that_gives_up_flags_the_call(sv, impatient, B, N, Hq, Hkv, D, page, lens):
    """Every status is written.  If a wait ran out anywhere, all of them say so, beside what is
    wrong with a request itself; if none did, the rows are right."""
    a = Attn(73, B, N, Hq, Hkv, D, page, lens, BF16)
    args, ws = list(a.args()), sv.AttentionWorkspace(B, N, Hq, Hkv, D, device="cuda")
    args[4] = i32([-1] + lens[1:])
    own = [sv.DEV_BAD_CACHE] + [0] * (B - 1)
    want, status = sv.tree_attention(*args)
    assert status.tolist() == own
    for ns in WAITS:
        for _ in range(5):
            out = torch.full_like(a.q, 7.0)
            status = impatient[ns](a, args, out, ws)
            if ns == 0 or status != own:
                assert status == [x | sv.DEV_TIMEOUT for x in own], ns
            else:
                assert torch.equal(out, want), ns


def test_attention_on_another_stream_and_in_a_graph(sv):
    a = Attn(41, 3, 6, 8, 2, 128, 32, [700, 12, 1500], BF16)
    want, _ = sv.tree_attention(*a.args())
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    args = a.args()
    side.wait_stream(torch.cuda.current_stream())
    got, _ = sv.tree_attention(*args, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    handle, _ = sv.tree_attention(*args, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(handle, want)
    ws = sv.AttentionWorkspace(3, 6, 8, 2, 128, device="cuda")
    out, status = torch.zeros_like(a.q), i32([9, 9, 9])
    graphs = []
    for _ in range(2):  # two graphs that take turns on one workspace
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            sv.tree_attention(*args, out=out, status=status, workspace=ws)
        graphs.append(g)
    for g in graphs + graphs:
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and status.tolist() == [0, 0, 0]


def test_attention_is_the_same_every_time(sv):
    a = Attn(43, 4, 16, 16, 2, 128, 64, [3000, 10, 777, 2048], BF16)
    first, _ = sv.tree_attention(*a.args())
    for _ in range(5):
        again, _ = sv.tree_attention(*a.args())
        assert torch.equal(first, again)


def test_attention_requests_that_share_pages(sv):
    """A common prompt's pages in two requests' tables, each with pages of its own behind them."""
    a = Attn(45, 2, 3, 4, 2, 64, 16, [64, 64], BF16)
    a.table[1, :4] = a.table[0, :4]
    a.check(sv)


def test_attention_whatever_the_workspace_holds(sv):
    a = Attn(47, 5, 20, 8, 2, 128, 64, [3000, 10, 777, 2048, 0], BF16)
    args, ws = a.args(), sv.AttentionWorkspace(5, 20, 8, 2, 128, device="cuda")
    want, _ = sv.tree_attention(*args)
    for fill in (0, 0xff, 0x7f, 1):
        ws.tensor.fill_(fill)
        got, status = sv.tree_attention(*args, workspace=ws)
        assert torch.equal(got, want) and status.tolist() == [0] * 5


@pytest.mark.parametrize("N,Hq,Hkv,lens", [
    (4, 4, 1, [30000]), (12, 8, 2, [9000]), (64, 4, 1, [20000]), (40, 16, 2, [7000, 12]),
])
def test_attention_few_items_of_many_pieces(sv, N, Hq, Hkv, lens):
    """One or a few items cut over all CTAs; on another stream and in a graph, over a workspace
    and an output that hold something else before each."""
    a = Attn(61, len(lens), N, Hq, Hkv, 128, 64, lens, BF16)
    args, ws = a.args(), sv.AttentionWorkspace(len(lens), N, Hq, Hkv, 128, device="cuda")
    parts, tol = a.want(many=True)
    out, side = torch.zeros_like(a.q), torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.tree_attention(*args, out=out, workspace=ws)
    first = None
    for run in (lambda: sv.tree_attention(*args, out=out, workspace=ws),
                lambda: sv.tree_attention(*args, out=out, workspace=ws, stream=side), g.replay):
        ws.tensor.fill_(0xff)
        out.fill_(7.0)
        torch.cuda.synchronize()
        run()
        torch.cuda.synchronize()
        for b in range(len(lens)):
            close(out[b], parts[0][b], tol[b], f"request {b}")
        assert first is None or torch.equal(out, first)
        first = out.clone()


@pytest.mark.parametrize("given", [True, False])
def test_attention_two_calls_at_once(sv, given):
    """On two streams, from two threads: a workspace each, given or made by the call."""
    import threading

    cases = [Attn(51, 6, 9, 8, 2, 128, 64, [900, 3000, 4, 77, 1500, 2], BF16),
             Attn(52, 3, 40, 16, 2, 64, 32, [2500, 1, 4000], F16)]
    wants = [sv.tree_attention(*a.args())[0] for a in cases]
    args = [a.args() for a in cases]
    spaces = [sv.AttentionWorkspace(a.B, a.N, a.q.shape[2], a.k.shape[2], a.D, device="cuda")
              if given else None for a in cases]
    torch.cuda.synchronize()
    outs, failures = [[], []], []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            for _ in range(30):
                outs[i].append(sv.tree_attention(*args[i], workspace=spaces[i], stream=stream)[0])
            stream.synchronize()
        except Exception as e:  # noqa: BLE001
            failures.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not failures
    for i in range(2):
        assert len(outs[i]) == 30 and all(torch.equal(o, wants[i]) for o in outs[i])


def test_attention_expanded_queries(sv):
    """Requests that share their queries (stride 0) and pages, with lengths of their own; an
    expanded page table, and an output without a place for every element, are refused."""
    a = Attn(53, 1, 4, 8, 2, 64, 32, [200], BF16)
    lens = i32([200, 131, 0])
    table, parents = a.table.repeat(3, 1), i32(np.repeat(a.parents, 3, 0))
    q = a.q.expand(3, -1, -1, -1)
    got, status = sv.tree_attention(q, a.k, a.v, table, lens, parents)
    assert status.tolist() == [0, 0, 0]
    parts = ref.attention(q, a.k, a.v, table, lens.tolist(), np.repeat(a.parents, 3, 0), [4] * 3, 64 ** -0.5)
    tol = ref.attention_tolerance(parts, 64, 204, BF16)
    for b in range(3):
        close(got[b], parts[0][b], tol[b], f"request {b}")
    with pytest.raises(sv.SpecVerifyError):
        sv.tree_attention(q, a.k, a.v, a.table.expand(3, -1), lens, parents)
    with pytest.raises(ValueError, match="place"):
        sv.tree_attention(q, a.k, a.v, table, lens, parents, out=torch.zeros_like(a.q).expand(3, -1, -1, -1))


# --------------------------------------------------------------------- append


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("B,N,Hq,Hkv,D,page,rot,interleaved,norm,chain,scale,layout", [
    (1, 1, 1, 1, 8, 16, 8, False, True, True, 1.0, "rows"),
    (2, 5, 32, 8, 128, 16, 128, False, True, True, 1.0, "rows"),
    (3, 32, 8, 2, 128, 64, 64, True, False, False, 1.0, "rows"),
    (2, 64, 4, 4, 64, 8, 32, False, True, False, 1.3, "heads"),
    (2, 7, 6, 2, 80, 24, 80, True, True, False, 1.0, "pairs"),
    (2, 9, 3, 1, 96, 1, 20, False, True, False, 0.7, "rows"),     # half a rotation inside a vector
    (1, 33, 4, 2, 120, 100, 6, True, False, False, 1.0, "rows"),  # pairs that end inside a vector
    (4, 3, 2, 1, 16, 3, 0, False, True, True, 1.0, "rows"),       # a norm without a rotation
    (1, 4, 2, 2, 128, 16, 0, False, False, True, 1.0, "rows"),    # an append alone
])
def test_append(sv, dtype, B, N, Hq, Hkv, D, page, rot, interleaved, norm, chain, scale, layout):
    rng = np.random.default_rng(N)
    lens = rng.integers(0, 300, B)
    nodes = rng.integers(1, N + 1, B)
    parents = None if chain else ref.random_parents(rng, B, N)
    k, v, table = ref.make_cache(3, B, N, Hkv, D, page, [int(x) for x in lens], dtype, "cuda",
                                 layout=layout, fill=7.0)
    k0, v0 = k.clone(), v.clone()
    qkv = torch.randn(B, N, (Hq + 2 * Hkv), D, device="cuda").to(dtype)
    q, kn, vn = qkv.split([Hq, Hkv, Hkv], 2)
    inv = f32(10000.0 ** (-np.arange(0, rot, 2) / max(rot, 1))) if rot else None
    qw, kw = ((1 + 0.2 * torch.randn(D, device="cuda")).to(dtype) if norm else None for _ in "qk")
    out = torch.full((B, N, Hq, D), 7.0, dtype=dtype, device="cuda")
    got, status = sv.append_nodes(q, kn, vn, k, v, table, i32(lens), inv,
                                  None if chain else i32(parents), i32(nodes), q_weight=qw,
                                  k_weight=kw, eps=1e-5, interleaved=interleaved, rope_scale=scale,
                                  q_out=out)
    torch.cuda.synchronize()
    assert got is out and status.tolist() == [0] * B
    want_k, want_v = k0.double(), v0.clone()
    tol_k = torch.zeros_like(want_k)
    for b in range(B):
        n = int(nodes[b])
        pos = torch.tensor([int(lens[b]) + len(ref.path_of(parents, b, i)) - 1 for i in range(n)],
                           device="cuda")
        want, size = ref.append(q[b, :n], pos, qw, 1e-5, inv, interleaved, scale)
        close(out[b, :n], want, ref.append_tolerance(want, size, dtype), "q")
        assert (out[b, n:] == 7.0).all()
        pg, off = ref.slots(table, b, page, list(range(lens[b], lens[b] + n)), "cuda")
        want, size = ref.append(kn[b, :n], pos, kw, 1e-5, inv, interleaved, scale)
        want_k[pg, off] = want
        tol_k[pg, off] = ref.append_tolerance(want, size, dtype)
        want_v[pg, off] = vn[b, :n]
    close(k, want_k, tol_k + 1e-30, "k")
    assert torch.equal(v, want_v)


def test_append_far_positions_and_in_place(sv):
    """Angles of positions near 2^20 and 2^30, where 32 bits lose them; q_out is q."""
    D, page = 64, 16
    inv = f32(500000.0 ** (-np.arange(0, D, 2) / D))
    for far in (2 ** 20 - 3, 2 ** 30 + 5):
        P = (far + 4) // page + 1
        table = torch.zeros(1, P, dtype=torch.int32, device="cuda")
        table[0, far // page] = 1
        table[0, (far + 3) // page] = 2 if (far + 3) // page != far // page else 1
        k, v = (torch.zeros(3, page, 1, D, dtype=BF16, device="cuda") for _ in "kv")
        q = torch.randn(1, 4, 2, D, device="cuda").to(BF16)
        kn, vn = (torch.randn(1, 4, 1, D, device="cuda").to(BF16) for _ in "kv")
        pos = torch.arange(far, far + 4, device="cuda")
        want, size = ref.append(q[0], pos, None, 0, inv, False, 1.0)
        got, status = sv.append_nodes(q, kn, vn, k, v, table, i32([far]), inv, q_out=q)
        assert got is q and status.tolist() == [0]
        close(q[0], want, ref.append_tolerance(want, size, BF16))
        pg, off = ref.slots(table, 0, page, list(range(far, far + 4)), "cuda")
        want, size = ref.append(kn[0], pos, None, 0, inv, False, 1.0)
        close(k[pg, off], want, ref.append_tolerance(want, size, BF16))
        assert torch.equal(v[pg, off], vn[0])


def test_append_keeps_odd_values(sv):
    """Infinities and NaN stay in their own heads; values are moved bit by bit."""
    k, v, table = ref.make_cache(1, 1, 2, 2, 64, 16, [3], BF16, "cuda", fill=0.0)
    q = torch.randn(1, 2, 2, 64, device="cuda").to(BF16)
    kn, vn = q.clone(), q.clone()
    q[0, 0, 0, 3] = float("inf")
    kn[0, 1, 1, 7] = float("nan")
    vn[0, 0, 0, 0] = float("nan")
    w = torch.ones(64, device="cuda", dtype=BF16)
    out, _ = sv.append_nodes(q, kn, vn, k, v, table, i32([3]), q_weight=w, k_weight=w)
    assert torch.isfinite(out[0, 0, 1]).all() and torch.isfinite(out[0, 1]).all()
    assert torch.isnan(out[0, 0, 0, 3])
    pg, off = ref.slots(table, 0, 16, [3, 4], "cuda")
    assert torch.isfinite(k[pg, off][0]).all() and torch.isfinite(k[pg, off][1, 0]).all()
    assert torch.isnan(k[pg, off][1, 1]).all()
    assert torch.equal(v[pg, off].view(torch.int16), vn[0].view(torch.int16))


def test_append_flags_bad_requests(sv):
    B, N = 5, 4
    k, v, table = ref.make_cache(2, B, N, 2, 64, 8, [30, 31, 32, 33, 34], BF16, "cuda", fill=7.0)
    q = torch.randn(B, N, 4, 64, device="cuda").to(BF16)
    kn, vn = (torch.randn(B, N, 2, 64, device="cuda").to(BF16) for _ in "kv")
    k0, v0 = k.clone(), v.clone()

    def call(nodes, lens, parents, pages):
        k.copy_(k0)
        v.copy_(v0)
        out = torch.full(q.shape, 7.0, dtype=BF16, device="cuda")
        got, status = sv.append_nodes(q, kn, vn, k, v, i32(pages), i32(lens), None, i32(parents),
                                      i32(nodes), q_out=out)
        if status[1] != 0:  # its cache rows stay
            own = table[1].long()
            assert torch.equal(k[own], k0[own]) and torch.equal(v[own], v0[own])
        return got, status

    _bad_requests(sv, call, table.cpu().numpy())


# ----------------------------------------------------------------------- keep


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("layers,B,N,Hkv,D,page,layout", [
    (1, 1, 1, 1, 8, 4, "rows"), (1, 4, 16, 2, 64, 16, "rows"), (3, 5, 64, 4, 128, 8, "rows"),
    (2, 3, 33, 3, 80, 5, "rows"), (1, 2, 20, 2, 64, 7, "heads"), (1, 2, 20, 2, 64, 7, "pairs"),
])
def test_keep_path(sv, dtype, layers, B, N, Hkv, D, page, layout):
    rng = np.random.default_rng(N)
    lens = rng.integers(0, 60, B)
    made = [ref.make_cache(9, B, N, Hkv, D, page, [int(x) for x in lens], dtype, "cuda",
                           layout=layout, fill=0.0) for _ in range(layers)]
    table = made[0][2]
    if layers == 1:
        k, v = made[0][0], made[0][1]
    else:
        k, v = torch.stack([m[0] for m in made]), torch.stack([m[1] for m in made])
    k.copy_(torch.randn(k.shape, device="cuda").to(dtype))
    v.copy_(torch.randn(v.shape, device="cuda").to(dtype))
    path, accepted = np.full((B, N), -1, np.int32), rng.integers(0, N, B)
    accepted[0] = N - 1  # the whole tree is a chain: every row stays
    for b in range(B):
        path[b, :accepted[b] + 1] = [0] + sorted(rng.choice(np.arange(1, N), accepted[b], replace=False))
    want = [k.clone(), v.clone()]
    for w, c in zip(want, (k, v)):
        w, c = (x if layers > 1 else x[None] for x in (w, c))
        for b in range(B):
            for j in range(1, accepted[b] + 1):
                (p0, o0), (p1, o1) = (ref.slots(table, b, page, [lens[b] + at], "cuda")
                                      for at in (path[b, j], j))
                w[:, p1, o1] = c[:, p0, o0]
    new, status = sv.keep_path(i32(path), i32(accepted), k, v, table, i32(lens))
    assert torch.equal(k, want[0]) and torch.equal(v, want[1])
    assert status.tolist() == [0] * B
    assert new.tolist() == (lens + accepted + 1).tolist()


def test_keep_flags_bad_requests(sv):
    B, N, page = 3, 6, 8
    lens = [20, 21, 22]
    k, v, table = ref.make_cache(2, B, N, 2, 64, page, lens, BF16, "cuda", fill=7.0)
    k0, v0 = k.clone(), v.clone()
    path = np.array([[0, 2, 5, -1, -1, -1]] * B)
    for change, bit in [
        (dict(accepted=-1), sv.DEV_BAD_DRAFT_LEN), (dict(accepted=N), sv.DEV_BAD_DRAFT_LEN),
        (dict(path=[1, 2, 5, -1, -1, -1]), sv.DEV_BAD_TREE),
        (dict(path=[0, 5, 5, -1, -1, -1]), sv.DEV_BAD_TREE),
        (dict(path=[0, 2, 6, -1, -1, -1]), sv.DEV_BAD_TREE),
        (dict(path=[0, -1, 2, -1, -1, -1]), sv.DEV_BAD_TREE),
        (dict(lens=-4), sv.DEV_BAD_CACHE), (dict(lens=2 ** 31 - 2), sv.DEV_BAD_CACHE),
        (dict(lens=page * table.shape[1] - 3), sv.DEV_BAD_CACHE),
        (dict(page=-1), sv.DEV_BAD_CACHE), (dict(page=10 ** 7), sv.DEV_BAD_CACHE),
    ]:
        k.copy_(k0)
        v.copy_(v0)
        p, ln, acc, t = path.copy(), list(lens), [2, 2, 2], table.clone()
        if "path" in change:
            p[1] = change["path"]
        if "lens" in change:
            ln[1] = change["lens"]
        if "accepted" in change:
            acc[1] = change["accepted"]
        if "page" in change:
            t[1, 23 // page] = change["page"]
        new, status = sv.keep_path(i32(p), i32(acc), k, v, t, i32(ln))
        assert status.tolist() == [0, bit, 0], change
        assert new.tolist() == [23, ln[1], 25]
        own = table[1].long()
        assert torch.equal(k[own].nan_to_num(0), k0[own].nan_to_num(0))
        assert torch.equal(v[own].nan_to_num(0), v0[own].nan_to_num(0))


# --------------------------------------------------------------------- logits


def _logits_case(seed, B, R, V, dtype, *, chain, L=64, nbias=0, mask=False, penalties=True,
                 ragged=True):
    rng = np.random.default_rng(seed)
    z = (3 * torch.randn(B, R, V, device="cuda",
                         generator=torch.Generator(device="cuda").manual_seed(seed))).to(dtype)
    history = (V * rng.random((B, L)) ** 2).astype(np.int32)
    seq = rng.integers(0, L + 1, B)
    prompt = (seq * rng.random(B)).astype(np.int64)
    tokens = (V * rng.random((B, R)) ** 4).astype(np.int32)
    d = dict(z=z, history=history, seq=seq, prompt=prompt,
             tokens=tokens[:, 1:] if chain else tokens,
             parents=None if chain else ref.random_parents(rng, B, R),
             nodes=rng.integers(1, R + 1, B) if ragged else np.full(B, R), ragged=ragged,
             rho=rng.uniform(0.8, 1.5, B).astype(np.float32) if penalties else None,
             freq=rng.uniform(-0.5, 1.0, B).astype(np.float32) if penalties else None,
             pres=rng.uniform(-0.5, 1.0, B).astype(np.float32) if penalties else None,
             bt=None, bv=None, allowed=None)
    if nbias:
        d["bt"] = rng.integers(0, V, (B, nbias)).astype(np.int32)
        d["bt"][:, ::7] = d["bt"][:, :1]  # the same token more than once
        d["bt"][:, 3::11] = -1
        d["bv"] = rng.uniform(-9, 9, (B, nbias)).astype(np.float32)
    if mask:
        d["allowed"] = rng.integers(-2 ** 31, 2 ** 31, (B, R, -(-V // 32))).astype(np.int32)
        d["allowed"][:, :, ::3] = 0
        d["allowed"][0, 0] = 0  # a row that allows nothing
    return d


def _logits_call(sv, d, **kw):
    put = lambda a, f=i32: None if a is None else f(a)  # noqa: E731
    return sv.process_logits(
        kw.pop("logits", d["z"]), i32(d["history"]), i32(d["seq"]), i32(d["prompt"]),
        tokens=i32(d["tokens"]), parents=put(d["parents"]),
        n_nodes=i32(d["nodes"]) if d["ragged"] else None, repetition=put(d["rho"], f32),
        frequency=put(d["freq"], f32), presence=put(d["pres"], f32), bias_tokens=put(d["bt"]),
        bias_values=put(d["bv"], f32), allowed=put(d["allowed"]), **kw)


def _logits_check(d, out):
    dtype = d["z"].dtype
    want, size = ref.logits(d["z"].float().cpu().numpy(), d["history"], d["seq"], d["prompt"],
                            d["tokens"], d["parents"], d["nodes"], d["rho"], d["freq"], d["pres"],
                            d["bt"], d["bv"], d["allowed"])
    tol = ref.logits_tolerance(want, size, dtype)
    for b in range(want.shape[0]):
        n = int(d["nodes"][b])
        close(out[b, :n], want[b, :n], tol[b, :n], f"request {b}")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,R,V,chain,kw", [
    (1, 1, 1, True, dict(L=4)),
    (1, 1, 31, True, dict(nbias=4, mask=True)),
    (2, 5, 1000, True, dict(L=200, nbias=30, mask=True)),
    (2, 5, 1024, False, dict(L=1, mask=True)),
    (3, 17, 4099, False, dict(L=333, nbias=12, mask=True)),   # rows of every alignment
    (2, 64, 2048, False, dict(L=2000, nbias=100)),
    (1, 64, 5000, True, dict(L=64, mask=True)),
    (2, 3, 33001, False, dict(L=5000, nbias=300, mask=True)),
    (2, 4, 32003, True, dict(penalties=False, mask=True)),
    (2, 4, 8192, True, dict(penalties=False, nbias=1024)),
    (65, 2, 777, True, dict(ragged=False)),
])
def test_logits(sv, dtype, B, R, V, chain, kw):
    d = _logits_case(V + R, B, R, V, dtype, chain=chain, **kw)
    out = torch.full_like(d["z"], 7.0)
    got, status = _logits_call(sv, d, out=out)
    torch.cuda.synchronize()
    assert got is out and status.tolist() == [0] * B
    _logits_check(d, out)
    for b in range(B):
        assert (out[b, int(d["nodes"][b]):] == 7.0).all()
    same = d["z"].clone()  # in place: the same bits, the rows behind the last untouched
    _logits_call(sv, d, logits=same, out=same)
    for b in range(B):
        n = int(d["nodes"][b])
        assert torch.equal(same[b, :n], out[b, :n]) and torch.equal(same[b, n:], d["z"][b, n:])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,R,V,chain,kw", [
    (76, 2, 777, True, dict(L=40, nbias=3, mask=True)),
    (80, 3, 8192, False, dict(L=100)),
    (30, 5, 20001, False, dict(L=300, nbias=9, mask=True)),   # rows of every alignment
    (10, 17, 65536, True, dict(L=3000, nbias=40, mask=True)),
    (8, 9, 100000, False, dict(L=700, penalties=False, mask=True)),
    (30, 2, 129280, True, dict(L=500, nbias=20, mask=True)),
    (58, 5, 65001, False, dict(L=600, nbias=7, mask=True)),
    (460, 1, 5000, True, dict(L=30000)),                      # a text that fills the lists
])
def test_logits_many_requests(sv, dtype, B, R, V, chain, kw):
    """Enough of them that blocks take large parts of the vocabulary."""
    d = _logits_case(V + B, B, R, V, dtype, chain=chain, **kw)
    out = torch.full_like(d["z"], 7.0)
    got, status = _logits_call(sv, d, out=out)
    assert got is out and status.tolist() == [0] * B
    _logits_check(d, out)
    for b in range(B):
        assert (out[b, int(d["nodes"][b]):] == 7.0).all()


def test_logits_expanded_inputs(sv):
    """Requests that share logits and a text (stride 0), each with penalties of its own."""
    d = _logits_case(12, 3, 4, 5001, BF16, chain=True, ragged=False)
    d["z"], d["history"] = d["z"][:1].repeat(3, 1, 1), np.repeat(d["history"][:1], 3, 0)
    want, _ = _logits_call(sv, d)
    text = i32(d["history"][:1]).expand(3, -1)
    got, status = sv.process_logits(
        d["z"][:1].expand(3, -1, -1), text, i32(d["seq"]), i32(d["prompt"]), tokens=i32(d["tokens"]),
        repetition=f32(d["rho"]), frequency=f32(d["freq"]), presence=f32(d["pres"]))
    assert status.tolist() == [0, 0, 0] and torch.equal(got, want)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_logits_strides_and_alignments(sv, dtype):
    """Rows inside wider ones, and an output that is aligned unlike the input."""
    d = _logits_case(5, 2, 4, 1001, dtype, chain=False, nbias=5, mask=True)
    want, _ = _logits_call(sv, d)
    wide = torch.zeros(2, 6, 1100, dtype=dtype, device="cuda")
    view = wide[:, 1:5, 3:1004]
    view.copy_(d["z"])
    for shift in (3, 4):
        room = torch.full((2, 5, 1100), 7.0, dtype=dtype, device="cuda")
        out = room[:, :4, shift:shift + 1001]
        _logits_call(sv, d, logits=view, out=out)
        for b in range(2):
            n = int(d["nodes"][b])
            assert torch.equal(out[b, :n], want[b, :n])
        out[:] = 7.0
        assert (room == 7.0).all()


def test_logits_two_dimensions_feed_the_sampler(sv):
    """One row a request: what sample_draft takes."""
    d = _logits_case(6, 9, 1, 3000, F32, chain=True, L=50, mask=True, ragged=False)
    d["allowed"][0, 0] = -1
    want, _ = _logits_call(sv, d)
    got, status = sv.process_logits(
        d["z"][:, 0], i32(d["history"]), i32(d["seq"]), i32(d["prompt"]), repetition=f32(d["rho"]),
        frequency=f32(d["freq"]), presence=f32(d["pres"]), allowed=i32(d["allowed"][:, 0]))
    assert torch.equal(got, want[:, 0]) and status.tolist() == [0] * 9
    tok = sv.sample_draft(got, f32(np.zeros(9)), f32(np.zeros(9)))
    assert torch.equal(tok.long(), got.argmax(-1))


def test_logits_odd_values(sv):
    """-inf, +inf and NaN logits: their own entries only; masked NaN becomes -inf."""
    z = torch.randn(1, 1, 64, device="cuda")
    z[0, 0, 3], z[0, 0, 4], z[0, 0, 5], z[0, 0, 6] = float("-inf"), float("inf"), float("nan"), float("nan")
    z[0, 0, 7] = torch.finfo(F32).min
    allowed = np.full((1, 1, 2), -1, np.int32)
    allowed[0, 0, 0] &= ~(1 << 6)
    out, _ = sv.process_logits(z, i32([[3, 4, 5, 6, 7]]), i32([5]), repetition=f32([2.0]),
                               presence=f32([1.0]), allowed=i32(allowed))
    got = out[0, 0].tolist()
    assert got[3] == float("-inf") and got[4] == float("inf") and np.isnan(got[5])
    assert got[6] == float("-inf") and got[7] == float("-inf")  # 2 * lowest
    assert torch.equal(out[0, 0, 8:], z[0, 0, 8:])


def test_logits_no_history(sv):
    z = torch.randn(2, 1, 100, device="cuda")
    out, status = sv.process_logits(z, torch.zeros(2, 0, dtype=torch.int32, device="cuda"), i32([0, 0]),
                                    repetition=f32([2.0, 2.0]))
    assert torch.equal(out, z) and status.tolist() == [0, 0]


def test_logits_one_token_all_over(sv):
    """Every token of a long text the same one: its count is exact."""
    z = torch.zeros(1, 2, 500, device="cuda")
    out, _ = sv.process_logits(z, i32(np.full((1, 30000), 123)), i32([30000]), tokens=i32([[123]]),
                               frequency=f32([0.5]))
    assert out[0, 0, 123] == -15000.0 and out[0, 1, 123] == -15000.5
    out[0, :, 123] = 0
    assert (out == 0).all()


def test_logits_flags_bad_requests(sv):
    B, R, V = 4, 3, 300
    d = _logits_case(7, B, R, V, F32, chain=False, L=40, nbias=4, ragged=False)
    d["seq"], d["prompt"], d["ragged"] = np.array([20] * B), np.array([5] * B), True
    clean, status = _logits_call(sv, d)
    assert status.tolist() == [0] * B
    for key, at, value, bit in [
        ("nodes", 2, 0, sv.DEV_BAD_DRAFT_LEN), ("nodes", 2, R + 1, sv.DEV_BAD_DRAFT_LEN),
        ("parents", (2, 1), 1, sv.DEV_BAD_TREE), ("tokens", (2, 2), V, sv.DEV_BAD_TOKEN),
        ("tokens", (2, 1), -1, sv.DEV_BAD_TOKEN), ("history", (2, 19), V, sv.DEV_BAD_TOKEN),
        ("history", (2, 0), -1, sv.DEV_BAD_TOKEN), ("seq", 2, 41, sv.DEV_BAD_CACHE),
        ("seq", 2, -1, sv.DEV_BAD_CACHE), ("prompt", 2, 21, sv.DEV_BAD_CACHE),
        ("prompt", 2, -1, sv.DEV_BAD_CACHE), ("rho", 2, 0.0, sv.DEV_BAD_PENALTY),
        ("rho", 2, float("nan"), sv.DEV_BAD_PENALTY), ("freq", 2, float("inf"), sv.DEV_BAD_PENALTY),
        ("pres", 2, float("nan"), sv.DEV_BAD_PENALTY), ("bt", (2, 0), V, sv.DEV_BAD_TOKEN),
    ]:
        bad = dict(d)
        bad[key] = d[key].copy()
        bad[key][at] = value
        out, status = _logits_call(sv, bad)
        assert status.tolist()[2] & bit and [s for i, s in enumerate(status.tolist()) if i != 2] == [0] * 3
        for b in (0, 1, 3):
            assert torch.equal(out[b], clean[b])
        assert (out[2] == float("-inf")).all()


def test_logits_on_another_stream_and_in_a_graph(sv):
    d = _logits_case(8, 3, 5, 4001, BF16, chain=True, nbias=3, mask=True, ragged=False)
    want, _ = _logits_call(sv, d)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        args = dict(history=i32(d["history"]), seq_lens=i32(d["seq"]), prompt_lens=i32(d["prompt"]),
                    tokens=i32(d["tokens"]), repetition=f32(d["rho"]), frequency=f32(d["freq"]),
                    presence=f32(d["pres"]), bias_tokens=i32(d["bt"]), bias_values=f32(d["bv"]),
                    allowed=i32(d["allowed"]))
    got, _ = sv.process_logits(d["z"], **args, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    out, status = torch.zeros_like(want), i32([5, 5, 5])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.process_logits(d["z"], **args, out=out, status=status)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and status.tolist() == [0, 0, 0]


def test_logits_two_calls_at_once(sv):
    """On two streams, from two threads, with texts whose lists take very different shared memory."""
    import threading

    cases = [_logits_case(81, 10, 2, 65536, BF16, chain=True, L=4, ragged=False),
             _logits_case(82, 10, 2, 65536, BF16, chain=True, L=9000, ragged=False)]
    wants, calls, failures = [], [], []
    for d in cases:
        want, _ = _logits_call(sv, d)
        wants.append(want)
        args = [d["z"], i32(d["history"]), i32(d["seq"]), i32(d["prompt"])]
        kw = dict(tokens=i32(d["tokens"]), repetition=f32(d["rho"]), frequency=f32(d["freq"]),
                  presence=f32(d["pres"]), out=torch.zeros_like(want), status=i32([9] * 10),
                  stream=torch.cuda.Stream())
        calls.append((args, kw))
    torch.cuda.synchronize()

    def work(args, kw):
        try:
            for _ in range(3000):
                sv.process_logits(*args, **kw)
            kw["stream"].synchronize()
        except Exception as e:  # noqa: BLE001
            failures.append(e)

    threads = [threading.Thread(target=work, args=c) for c in calls]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not failures
    for (_, kw), want in zip(calls, wants):
        assert torch.equal(kw["out"], want) and kw["status"].tolist() == [0] * 10


# ------------------------------------------------------------------- together


def test_a_tree_step_from_projection_to_kept_rows(sv):
    """Three steps of one layer: append, attend, penalise, verify, keep, insert.
    The cache that the tree steps leave is the one that a plain run of the
    accepted tokens makes, and the attention agrees with the 64-bit form."""
    rng = np.random.default_rng(0)
    B, N, Hq, Hkv, D, page, V, L = 3, 12, 4, 2, 64, 8, 512, 200
    lens = [17, 40, 0]
    k, v, table = ref.make_cache(4, B, 64, Hkv, D, page, lens, BF16, "cuda", fill=0.0)
    history = rng.integers(0, V, (B, L)).astype(np.int32)
    hist_t, seq_t = i32(history), i32([n + 1 for n in lens])
    cache_lens = i32(lens)
    inv = f32(10000.0 ** (-np.arange(0, D, 2) / D))
    w = torch.ones(D, device="cuda", dtype=BF16)
    rho = f32([1.2, 1.0, 1.4])
    for step in range(3):
        parents, nodes = ref.random_parents(rng, B, N), rng.integers(4, N + 1, B)
        qkv = torch.randn(B, N, Hq + 2 * Hkv, D, device="cuda").to(BF16)
        q, kn, vn = qkv.split([Hq, Hkv, Hkv], 2)
        before = cache_lens.tolist()
        pt, nt = i32(parents), i32(nodes)
        q_rot, s1 = sv.append_nodes(q, kn, vn, k, v, table, cache_lens, inv, pt, nt, q_weight=w,
                                    k_weight=w)
        out, s2 = sv.tree_attention(q_rot, k, v, table, cache_lens, pt, nt)
        parts = ref.attention(q_rot, k, v, table, before, parents, nodes, D ** -0.5)
        tol = ref.attention_tolerance(parts, D, max(before) + N, BF16)
        for b in range(B):
            n = int(nodes[b])
            close(out[b, :n], parts[0][b, :n], tol[b, :n])
        logits = torch.randn(B, N, V, device="cuda")
        tokens = rng.integers(0, V, (B, N)).astype(np.int32)
        for b in range(B):  # the draft proposes what the target says for some nodes
            for i in range(1, int(nodes[b])):
                if rng.random() < 0.8:
                    logits[b, parents[b, i], tokens[b, i]] = 9.0 + i
        fixed, s3 = sv.process_logits(logits, hist_t, seq_t, tokens=i32(tokens), parents=pt,
                                      n_nodes=nt, repetition=rho)
        acc, toks, path = sv.verify_tree_greedy(fixed, pt, i32(tokens), nt)
        new_lens, s4 = sv.keep_path(path, acc, k, v, table, cache_lens)
        torch.cuda.synchronize()
        for s in (s1, s2, s3, s4):
            assert s.tolist() == [0] * B
        assert (acc >= 0).all()
        for b in range(B):
            A = int(acc[b])
            assert new_lens[b] == before[b] + A + 1
            nodes_kept = path[b, :A + 1].long()
            pg, off = ref.slots(table, b, page, list(range(before[b], before[b] + A + 1)), "cuda")
            assert torch.equal(v[pg, off], vn[b, nodes_kept])
            pos = torch.arange(before[b], before[b] + A + 1, device="cuda")
            want, size = ref.append(kn[b, nodes_kept], pos, w, 1e-6, inv, False, 1.0)
            close(k[pg, off], want, ref.append_tolerance(want, size, BF16))
        sv.insert_accepted(acc, toks, seq_t, hist_t)
        cache_lens = new_lens
