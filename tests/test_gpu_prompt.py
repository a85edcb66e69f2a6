"""The prompt's pass over the paged cache against plain 64-bit forms: the append
of a ragged batch's projections and the attention of its tokens."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import prompt_reference as ref  # noqa: E402
import tree_reference as tree  # noqa: E402
from test_gpu_tree import BF16, F16, close, f32, i32, sv  # noqa: E402, F401

pytestmark = pytest.mark.gpu


class Attn:
    """One call's inputs: requests of new[b] tokens behind lens[b] cached ones.  Places of the
    cache that no token has hold NaN; with a window, pages that nobody sees do not exist."""

    def __init__(self, seed, new, lens, Hq, Hkv, D, page, dtype, *, cap=None, window=None, prefix=None,
                 slopes=False, scale=None, layout="rows", sharp=1.0, spare=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.new, self.lens, self.dtype, self.D, self.page = new, lens, dtype, D, page
        self.Hq, self.Hkv, self.B = Hq, Hkv, len(new)
        self.cu = np.concatenate([[0], np.cumsum(new)])
        T = int(self.cu[-1]) + spare  # spare: rows of no request
        total = [a + b for a, b in zip(lens, new)]
        self.k, self.v, self.table = tree.make_cache(seed, self.B, 1, Hkv, D, page, total, dtype, "cuda",
                                                     layout=layout)
        self.q = (sharp * torch.randn(T, Hq, D, generator=gen, device="cuda")).to(dtype)
        self.cap, self.window, self.scale = cap, window, scale
        self.prefix = None if prefix is None else list(prefix)
        self.slopes = 2.0 ** -(1.0 + torch.arange(Hq, device="cuda") * 7 / Hq) if slopes else None
        if window is not None:
            for b in range(self.B):
                below = max(0, lens[b] - window + 1)
                kept = self.prefix[b] if self.prefix else 0
                for p in range(-(-kept // page), below // page):
                    self.table[b, p] = -1 - p

    def args(self):
        return self.q, self.k, self.v, self.table, i32(self.lens), i32(self.cu)

    def kw(self):
        return dict(cap=self.cap, window=self.window, slopes=self.slopes, scale=self.scale,
                    prefix_lens=None if self.prefix is None else i32(self.prefix))

    def want(self):
        return ref.attention(self.q, self.k, self.v, self.table, self.lens, self.cu,
                             self.scale or self.D ** -0.5, self.cap, self.window, self.prefix, self.slopes)

    def check(self, sv, **kw):
        out = torch.full(self.q.shape, 7.0, dtype=self.dtype, device="cuda")
        got, status = sv.chunk_attention(*self.args(), out=out, **self.kw(), **kw)
        torch.cuda.synchronize()
        assert got is out and status.tolist() == [0] * self.B
        want, tol = self.want()
        n = int(self.cu[-1])
        close(got[:n], want[:n], tol[:n])
        assert (got[n:] == 7.0).all()  # rows of no request


SHAPES = [  # new, lens, Hq, Hkv, D, page
    ([1], [0], 1, 1, 8, 16),
    ([1], [1], 8, 8, 64, 16),
    ([1, 1], [127, 128], 8, 1, 128, 16),
    ([3, 0, 1], [0, 5, 129], 12, 4, 128, 64),
    ([64], [0], 8, 4, 128, 32),                 # 128 rows exactly
    ([65], [63], 8, 4, 128, 32),                # and one token more
    ([128, 129], [0, 1], 4, 2, 64, 128),        # 256 rows, 258
    ([300], [17], 2, 2, 64, 64),                # a key head to each query head
    ([37, 200, 1, 90], [300, 0, 777, 31], 14, 2, 128, 16),   # groups of seven
    ([50], [333], 7, 1, 80, 24),
    ([9, 140], [5, 140], 9, 3, 96, 1),          # a page to each slot
    ([100], [513], 4, 4, 120, 100),
    ([33, 2], [77, 0], 10, 2, 24, 3),
    ([260], [900], 64, 4, 112, 200),
    ([2, 1, 2, 1], [3, 0, 254, 126], 2, 2, 40, 8),
    ([700], [1], 16, 1, 128, 64),               # sixteen rows to a token
]
MODS = [
    dict(),
    dict(cap=4.0),
    dict(slopes=True),
    dict(window=1),
    dict(window=100, prefix=4),
    dict(window=7, prefix=150, cap=30.0, slopes=True),
    dict(prefix=40, slopes=True),
    dict(prefix=10 ** 6),                       # all of it, the tokens behind too
]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
@pytest.mark.parametrize("mod", range(len(MODS)))
def test_attention(sv, dtype, shape, mod):  # noqa: F811
    new, lens, Hq, Hkv, D, page = SHAPES[shape]
    kw = dict(MODS[mod])
    if "prefix" in kw:
        kw["prefix"] = [max(0, kw["prefix"] - b) for b in range(len(new))]
    Attn(31 * shape + mod, new, lens, Hq, Hkv, D, page, dtype, spare=2 * (shape % 2), **kw).check(
        sv, longest=max(new) if mod % 2 else None)


SINGLES = [  # new, lens, Hq, Hkv, D, page: no request with more than one token
    ([1], [0], 1, 1, 8, 16),
    ([1, 0, 1], [1, 70, 63], 16, 1, 128, 16),        # sixteen rows, 64 slots
    ([1, 1], [64, 511], 17, 1, 64, 8),               # one row more than the small kernel takes
    ([1, 1, 1], [4001, 0, 2500], 32, 8, 128, 16),
    ([1], [4001], 32, 8, 128, 16),
    ([1], [8191], 16, 4, 64, 32),
    ([0, 1, 1], [5, 999, 513], 14, 2, 80, 24),
    ([1, 1], [3000, 130], 6, 3, 96, 1),
    ([1] * 5, [40, 700, 5, 1, 3000], 9, 3, 24, 100),
    ([1, 1], [7000, 12], 8, 8, 112, 64),
    ([1, 1], [777, 63], 11, 1, 40, 7),
]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("shape", range(len(SINGLES)))
@pytest.mark.parametrize("mod", range(len(MODS)))
def test_attention_single_tokens(sv, dtype, shape, mod):  # noqa: F811
    new, lens, Hq, Hkv, D, page = SINGLES[shape]
    kw = dict(MODS[mod])
    if "prefix" in kw:
        kw["prefix"] = [max(0, kw["prefix"] - b) for b in range(len(new))]
    Attn(37 * shape + mod, new, lens, Hq, Hkv, D, page, dtype, spare=2 * (shape % 2), **kw).check(sv, longest=1)


@pytest.mark.parametrize("layout", ["heads", "pairs"])
def test_attention_single_tokens_of_many_requests(sv, layout):  # noqa: F811
    """Clusters of eight CTAs, of four and of two, and more requests than the small kernel takes."""
    rng = np.random.default_rng(4)
    for B, most in ((8, 900), (16, 900), (38, 700), (39, 700), (700, 150)):
        new, lens = [int(x) for x in rng.integers(0, 2, B)], [int(x) for x in rng.integers(0, most, B)]
        Attn(B, new, lens, 8, 2, 64, 16, F16, window=200, prefix=[3] * B, layout=layout).check(sv, longest=1)


def test_attention_single_tokens_flagged_and_repeated(sv):  # noqa: F811
    a = Attn(79, [1, 1, 1, 1], [300, 40, 900, 12], 8, 2, 128, 16, BF16, window=500)
    args = a.args()
    want, status = sv.chunk_attention(*args, longest=1, **a.kw())
    assert status.tolist() == [0] * 4

    def call(lens=a.lens, cu=a.cu, table=a.table):
        out = torch.full_like(a.q, 7.0)
        _, status = sv.chunk_attention(a.q, a.k, a.v, table, i32(lens), i32(cu), window=500, longest=1, out=out)
        return out, status.tolist()

    for bad_page in (-1, 10 ** 6, 2 ** 31 - 1):
        for at in (401 // 16, 900 // 16):  # the window's first page, and the last
            table = a.table.clone()
            table[2, at] = bad_page
            out, status = call(table=table)
            assert status == [0, 0, sv.DEV_BAD_CACHE, 0] and (out[2] == 0).all()
            assert torch.equal(out[[0, 1, 3]], want[[0, 1, 3]])
    for lens in ([300, -1, 900, 12], [300, 10 ** 6, 900, 12], [300, 2 ** 31 - 1, 900, 12]):
        out, status = call(lens=lens)
        assert status == [0, sv.DEV_BAD_CACHE, 0, 0] and (out[1] == 0).all()
        assert torch.equal(out[[0, 2, 3]], want[[0, 2, 3]])
    out, status = call(cu=[0, 1, 3, 4, 4])  # two tokens where one was said
    assert status == [0, sv.DEV_BAD_DRAFT_LEN, 0, 0] and (out[1:3] == 0).all() and torch.equal(out[0], want[0])
    out, status = call(cu=[0, 1, 10 ** 6, 3, 4])
    assert status == [0, sv.DEV_BAD_DRAFT_LEN, sv.DEV_BAD_DRAFT_LEN, 0] and (out[1:3] == 7.0).all()
    # the same on another stream, and in a graph over other lengths
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, _ = sv.chunk_attention(*args, longest=1, stream=side, **a.kw())
    side.synchronize()
    assert torch.equal(got, want)
    out, status = torch.zeros_like(a.q), i32([9] * 4)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.chunk_attention(*args, longest=1, out=out, status=status, window=500)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and status.tolist() == [0] * 4
    args[4].copy_(i32([100, 20, 900, 2]))  # places that hold values, pages that exist
    g.replay()
    torch.cuda.synchronize()
    fresh, status = sv.chunk_attention(*args, longest=1, window=500)
    assert torch.equal(out, fresh) and status.tolist() == [0] * 4


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_attention_single_tokens_hidden_places_hold_anything(sv, bad):  # noqa: F811
    a = Attn(83, [1, 1], [90, 333], 4, 2, 64, 32, BF16, window=70, prefix=[5, 40])
    for b, slots in ((0, (6, 20, 21)), (1, (41, 200, 263))):  # behind the prefix, before the window
        for at in slots:
            page = a.table[b, at // 32]
            if page >= 0:
                a.k[page.long(), at % 32] = bad
                a.v[page.long(), at % 32] = bad
    a.check(sv, longest=1)
    at = 333  # its own: seen
    a.v[a.table[1, at // 32].long(), at % 32, 0, 3] = bad
    a.check(sv, longest=1)


@pytest.mark.parametrize("page", [2, 12, 40, 48, 96, 136, 384])
@pytest.mark.parametrize("layout", ["rows", "heads", "pairs"])
def test_attention_pages_and_layouts(sv, page, layout):  # noqa: F811
    Attn(page, [70, 5], [400, 130], 4, 2, 64, page, BF16, layout=layout, window=200, prefix=[9, 0]).check(sv)


@pytest.mark.parametrize("kw", [dict(), dict(window=600, prefix=[5, 700, 0]), dict(cap=2.0, slopes=True)])
@pytest.mark.parametrize("dtype,new,lens,Hq,Hkv,D,page", [
    (BF16, [1, 1, 1], [9000, 3, 2999], 4, 1, 128, 64),          # single tokens: split over the keys
    (F16, [2, 1, 40], [5000, 0, 4097], 16, 2, 128, 32),
    (BF16, [1500, 777, 1], [0, 2000, 5000], 8, 2, 128, 64),     # runs that cut items in the middle
    (F16, [1023, 1, 513], [1, 3000, 100], 4, 4, 64, 16),
])
def test_attention_long(sv, kw, dtype, new, lens, Hq, Hkv, D, page):  # noqa: F811
    Attn(5, new, lens, Hq, Hkv, D, page, dtype, **kw).check(sv, longest=max(new))


def test_attention_many_requests(sv):  # noqa: F811
    rng = np.random.default_rng(3)
    new = [int(x) for x in rng.integers(0, 6, 700)]
    lens = [int(x) for x in rng.integers(0, 300, 700)]
    Attn(7, new, lens, 2, 1, 32, 16, BF16, window=90).check(sv, longest=5)


@pytest.mark.parametrize("sharp", [0.0, 20.0])
@pytest.mark.parametrize("cap", [None, 50.0])
def test_attention_flat_and_sharp_scores(sv, sharp, cap):  # noqa: F811
    Attn(13, [200, 3], [300, 900], 8, 2, 128, 64, F16, sharp=sharp, cap=cap).check(sv)


@pytest.mark.parametrize("longest", [1, 70])
@pytest.mark.parametrize("cap", [0.5, 8.0, 1000.0, 1e6])
def test_attention_caps(sv, cap, longest):  # noqa: F811
    """Scores far below the cap, about it and far above; a large cap costs no precision."""
    a = Attn(19, [1, 1] if longest == 1 else [70, 1], [300, 901], 4, 2, 64, 32, F16, sharp=3.0, cap=cap)
    at = 120  # one key much larger than all others, which sees only few scores near the cap
    a.k[a.table[0, at // 32].long(), at % 32] *= 40
    a.check(sv, longest=longest)
    want, _ = a.want()
    got, _ = sv.chunk_attention(*a.args(), longest=longest, **a.kw())
    rel = ((got.double() - want).norm() / want.norm()).item()
    # the output's and the weights' roundings to f16, 2^-11 of a value each, with half as much again
    assert rel < 1.5 * 2.0 ** -10, rel


@pytest.mark.parametrize("slopes", [False, True])
@pytest.mark.parametrize("longest", [1, 70])
@pytest.mark.parametrize("cap", [1e-29, 1e9, 1e15, 1e21, 1e25, 1e29])
def test_attention_caps_of_any_size(sv, cap, longest, slopes):  # noqa: F811
    """A cap far above all scores leaves them as they are: cap tanh(y / cap) is y (1 - (y / cap)^2 / 3).  For
    these y below 300 it is less than 2^-40 of it, and the kernels' form of it is off by the
    polynomial's 2^-23.7 and four roundings, together below 2^-21 of y: the tolerance of an
    attention without caps has it among the 2^-19 that it gives to a score beside its D sums.  A cap far
    below them makes all weights alike."""
    a = Attn(101, [1, 1] if longest == 1 else [70, 1], [300, 901], 4, 2, 64, 32, F16, sharp=3.0, slopes=slopes)
    if cap < 1.0:
        a.cap = cap
    want, tol = a.want()
    a.cap = cap
    got, status = sv.chunk_attention(*a.args(), longest=longest, **a.kw())
    assert status.tolist() == [0, 0]
    close(got, want, tol)
    rel = ((got.double() - want).norm() / want.norm()).item()
    # the output's and the weights' roundings to f16, 2^-11 of a value each, with half as much again
    assert rel < 1.5 * 2.0 ** -10, rel


def test_attention_rising_maxima(sv):  # noqa: F811
    """Every tile has larger scores than the one before, so every one scales the sums again."""
    a = Attn(17, [150], [1000], 2, 2, 64, 32, BF16, scale=1.0)
    pos = torch.arange(1150, device="cuda")
    pg, off = a.table[0].long()[pos // 32], pos % 32
    a.k[pg, off] = 0.0
    a.k[pg, off, :, 0] = (pos // 16).to(BF16)[:, None]
    a.q.zero_()
    a.q[:, :, 0] = 1.0
    a.check(sv)
    a.k[pg, off, :, 0] = -(pos // 16).to(BF16)[:, None]
    a.check(sv)


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("new,Hq,window,prefix", [
    ([20], 2, None, None), ([200], 4, None, None), ([300], 2, 130, None), ([300], 2, 40, [60]), ([150], 8, 1, None),
])
def test_attention_hidden_values_hold_anything(sv, bad, new, Hq, window, prefix):  # noqa: F811
    """A value that is not finite reaches the tokens that see its slot, and no other."""
    a = Attn(23, new, [77], Hq, 1, 64, 32, BF16, window=window, prefix=prefix)
    for at in (76, 77, 80, 77 + new[0] // 2, 77 + new[0] - 1, 30):
        page = a.table[0, at // 32]
        if page >= 0:
            a.v[page.long(), at % 32, 0, at % 64] = bad
    a.check(sv)


def test_attention_hidden_keys_hold_anything(sv):  # noqa: F811
    """A key of NaN makes its own tokens' rows NaN, not those that do not see it."""
    a = Attn(29, [130], [50], 4, 2, 64, 32, F16, window=64, cap=10.0, slopes=True)
    clean, _ = sv.chunk_attention(*a.args(), **a.kw())
    at = 50 + 70
    a.k[a.table[0, at // 32].long(), at % 32, 1] = float("nan")
    got, status = sv.chunk_attention(*a.args(), **a.kw())
    assert status.tolist() == [0]
    sees = torch.arange(130, device="cuda")
    sees = (sees >= 70) & (sees < 70 + 64)
    assert torch.equal(got[~sees], clean[~sees])
    assert torch.equal(got[:, :2], clean[:, :2])  # the other key head's
    assert torch.isnan(got[sees][:, 2:]).all()


def test_attention_masks_of_the_lowest_values(sv):  # noqa: F811
    """Keys so far down that their scores are -inf or the type's lowest count nothing."""
    a = Attn(37, [40], [200], 2, 2, 64, 64, BF16, scale=1.0)
    a.q.fill_(1.0)
    pos = torch.arange(0, 200, 3, device="cuda")
    a.k[a.table[0].long()[pos // 64], pos % 64] = -3e38 / 64
    a.check(sv)


def test_attention_strided_queries_and_outputs(sv):  # noqa: F811
    a = Attn(41, [50, 7], [90, 300], 8, 2, 64, 16, BF16)
    want, _ = sv.chunk_attention(*a.args(), **a.kw())
    qkv = torch.zeros(57, 12 * 64, dtype=BF16, device="cuda")
    qkv[:, :512] = a.q.flatten(1)
    wide = torch.zeros(8, 57, 72, dtype=BF16, device="cuda").transpose(0, 1)
    a.q = qkv[:, :512].unflatten(1, (8, 64))
    out, _ = sv.chunk_attention(*a.args(), out=wide[..., :64], **a.kw())
    assert torch.equal(out, want) and (wide[..., 64:] == 0).all()
    a.q = want[:1].expand(57, 8, 64)  # a query for all
    same, _ = sv.chunk_attention(*a.args(), **a.kw())
    a.q = want[:1].expand(57, 8, 64).contiguous()
    assert torch.equal(same, sv.chunk_attention(*a.args(), **a.kw())[0])


def test_attention_offsets_past_32_bits(sv):  # noqa: F811
    """Pages 2^31 elements and more into the cache."""
    a = Attn(43, [30], [100], 4, 2, 64, 16, BF16)
    want, _ = sv.chunk_attention(*a.args(), **a.kw())
    stride = 2 ** 29  # elements from page to page: the last begins at 2^32
    far = []
    for c in (a.k, a.v):
        wide = torch.empty(9 * stride, dtype=BF16, device="cuda").as_strided((9, 16, 2, 64), (stride, 128, 64, 1))
        for p in range(9):
            wide[p] = c[a.table[0, p].long()]
        far.append(wide)
    a.k, a.v = far
    a.table = i32(np.arange(9)[None])
    got, status = sv.chunk_attention(*a.args(), **a.kw())
    assert status.tolist() == [0] and torch.equal(got, want)


def test_attention_flags_bad_requests(sv):  # noqa: F811
    new, lens = [20, 30, 9, 14, 1], [100, 40, 70, 0, 12]
    a = Attn(47, new, lens, 4, 2, 64, 16, BF16, prefix=[3, 0, 5, 0, 0])
    want, _ = sv.chunk_attention(*a.args(), **a.kw())
    cu, table = a.cu, a.table.clone()

    def call(lens=lens, cu=cu, table=table, prefix=a.prefix, **kw):
        out = torch.full_like(a.q, 7.0)
        _, status = sv.chunk_attention(a.q, a.k, a.v, table, i32(lens), i32(cu), prefix_lens=i32(prefix),
                                       out=out, **kw)
        return out, status.tolist()

    def others(out, bad, value):
        for b in range(5):
            rows = slice(int(cu[b]), int(cu[b + 1]))
            assert torch.equal(out[rows], want[rows]) if b != bad else (out[rows] == value).all(), b

    out, status = call(lens=[100, -1, 70, 0, 12])
    assert status == [0, sv.DEV_BAD_CACHE, 0, 0, 0]
    others(out, 1, 0.0)
    out, status = call(lens=[100, 40, 10 ** 6, 0, 12])
    assert status == [0, 0, sv.DEV_BAD_CACHE, 0, 0]
    others(out, 2, 0.0)
    out, status = call(lens=[100, 40, 70, 2 ** 31 - 5, 12])
    assert status == [0, 0, 0, sv.DEV_BAD_CACHE, 0]
    others(out, 3, 0.0)
    out, status = call(prefix=[3, -1, 5, 0, 0])
    assert status == [0, sv.DEV_BAD_CACHE, 0, 0, 0]
    others(out, 1, 0.0)
    out, status = call(longest=29)  # request 1 has 30
    assert status == [0, sv.DEV_BAD_DRAFT_LEN, 0, 0, 0]
    others(out, 1, 0.0)
    for page in (-1, 10 ** 6, 2 ** 31 - 1):
        for at in (0, 2, 4):
            bad = table.clone()
            bad[1, at] = page
            out, status = call(table=bad)
            assert status == [0, sv.DEV_BAD_CACHE, 0, 0, 0]
            others(out, 1, 0.0)
    # cu_tokens that falls, or leaves the rows: the request has no rows
    fall = cu.copy()
    fall[4] = 10 ** 6
    out, status = call(cu=fall)
    assert status[:3] == [0, 0, 0] and status[3] & status[4] & sv.DEV_BAD_DRAFT_LEN
    assert torch.equal(out[:int(cu[3])], want[:int(cu[3])]) and (out[int(cu[3]):] == 7.0).all()
    out, status = call(cu=[0, 20, 10, 10, 10, 11])
    assert status[1] == sv.DEV_BAD_DRAFT_LEN
    out, status = call(cu=[-5, 20, 50, 59, 73, 74])
    assert status == [sv.DEV_BAD_DRAFT_LEN, 0, 0, 0, 0] and (out[:20] == 7.0).all()
    assert torch.equal(out[20:], want[20:])


def test_attention_no_tokens(sv):  # noqa: F811
    a = Attn(53, [0, 0], [10, 20], 4, 2, 64, 16, BF16)
    out, status = sv.chunk_attention(*a.args(), **a.kw())
    assert out.shape == (0, 4, 64) and status.tolist() == [0, 0]
    spare = torch.full((3, 4, 64), 7.0, dtype=BF16, device="cuda")
    _, status = sv.chunk_attention(torch.zeros_like(spare), *a.args()[1:], out=spare)
    assert status.tolist() == [0, 0] and (spare == 7.0).all()


def test_attention_is_a_chunk_of_the_whole(sv):  # noqa: F811
    """A prompt in one call or in chunks, and its last token alone as tree_attention has it."""
    a = Attn(59, [500], [0], 8, 2, 128, 64, BF16)
    (want, tol), whole = a.want(), sv.chunk_attention(*a.args())[0]
    close(whole, want, tol)
    for first, last in [(0, 100), (100, 101), (101, 385), (385, 500)]:
        part, _ = sv.chunk_attention(a.q[first:last], a.k, a.v, a.table, i32([first]), i32([0, last - first]))
        close(part, want[first:last], tol[first:last])
    alone, _ = sv.tree_attention(a.q[None, 499:], a.k, a.v, a.table, i32([499]))
    close(alone[0], want[499:], tol[499:])


def test_attention_on_another_stream_and_in_a_graph(sv):  # noqa: F811
    a = Attn(61, [300, 1, 40], [700, 12, 1500], 8, 2, 128, 32, BF16, window=900, cap=20.0)
    args, kw = a.args(), a.kw()
    want, _ = sv.chunk_attention(*args, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream):
        got, _ = sv.chunk_attention(*args, stream=stream, **kw)
        side.synchronize()
        assert torch.equal(got, want)
    ws = sv.ChunkWorkspace(300, 8, 2, 128, device="cuda")
    out, status = torch.zeros_like(a.q), i32([9, 9, 9])
    graphs = []
    for _ in range(2):  # two graphs that take turns on one workspace
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            sv.chunk_attention(*args, out=out, status=status, workspace=ws, longest=300, **kw)
        graphs.append(g)
    for g in graphs + graphs:
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and status.tolist() == [0, 0, 0]
    # other contents of the same places: fewer tokens, another length
    args[4].copy_(i32([400, 100, 5]))
    args[5].copy_(i32([0, 10, 10, 250]))
    graphs[0].replay()
    torch.cuda.synchronize()
    fresh, _ = sv.chunk_attention(*args, longest=300, **kw)
    assert torch.equal(out[:250], fresh[:250])


def test_attention_is_the_same_every_time(sv):  # noqa: F811
    a = Attn(67, [300, 1, 777], [3000, 10, 48], 16, 2, 128, 64, BF16, slopes=True)
    first, _ = sv.chunk_attention(*a.args(), **a.kw())
    for fill in (0, 255, 127):
        ws = sv.ChunkWorkspace(1078, 16, 2, 128, device="cuda")
        ws.tensor.fill_(fill)  # whatever the workspace holds
        again, _ = sv.chunk_attention(*a.args(), workspace=ws, **a.kw())
        assert torch.equal(again, first)


def test_attention_two_calls_at_once(sv):  # noqa: F811
    cases = [Attn(71 + i, [400 + i, 3], [1000, 5000 * i], 8, 2, 128, 64, BF16) for i in range(2)]
    want = [sv.chunk_attention(*c.args())[0] for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    ws = [sv.ChunkWorkspace(500, 8, 2, 128, device="cuda") for _ in cases]
    args, outs = [c.args() for c in cases], [torch.zeros_like(c.q) for c in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, a, o, w in zip(streams, args, outs, ws):
            sv.chunk_attention(*a, out=o, workspace=w, longest=500, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_workspace_too_small(sv):  # noqa: F811
    a = Attn(73, [40], [10], 8, 2, 64, 16, BF16)
    with pytest.raises(sv.SpecVerifyError):
        sv.chunk_attention(*a.args(), workspace=sv.ChunkWorkspace(1, 8, 2, 64, device="cuda"))


# --------------------------------------------------------------------- append


def run_append(sv, seed, new, lens, Hq, Hkv, D, page, dtype, *, axes, rot, interleaved, norm, scale,  # noqa: F811
               layout="rows", spare=0, in_place=False, far=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    B, cu = len(new), np.concatenate([[0], np.cumsum(new)])
    T = int(cu[-1]) + spare
    k_cache, v_cache, table = tree.make_cache(seed, B, max(new) if new else 1, Hkv, D, page, lens, dtype, "cuda",
                                              layout=layout)
    k_was, v_was = k_cache.clone(), v_cache.clone()
    qkv = torch.randn(T, (Hq + 2 * Hkv) * D, generator=gen, device="cuda").to(dtype)
    q, k, v = (x.unflatten(-1, (-1, D)) for x in qkv.split([Hq * D, Hkv * D, Hkv * D], -1))
    half = rot // 2
    freq = 10000.0 ** (-torch.arange(half, device="cuda") / max(half, 1)) if half else None
    positions = axis_of = None
    if axes and half:
        positions = torch.randint(-5, 100000, (axes, T), generator=gen, device="cuda", dtype=torch.int32) + far
        axis_of = torch.randint(0, axes, (half,), generator=gen, device="cuda", dtype=torch.int32)
    weights = [(1 + 0.2 * torch.randn(D, generator=gen, device="cuda")).to(dtype) if norm else None for _ in "qk"]
    was = q.clone()
    q_out = q if in_place else torch.full((T, Hq, D), 7.0, dtype=dtype, device="cuda")
    got, status = sv.append_chunk(q, k, v, k_cache, v_cache, table, i32(lens), i32(cu), freq,
                                  positions=positions, axis_of=axis_of, q_weight=weights[0],
                                  k_weight=weights[1], eps=1e-5, interleaved=interleaved, rope_scale=scale,
                                  q_out=q_out)
    torch.cuda.synchronize()
    assert got is q_out and status.tolist() == [0] * B
    used_k, used_v = k_was, v_was
    for b in range(B):
        rows = slice(int(cu[b]), int(cu[b + 1]))
        n = new[b]
        slot = torch.arange(lens[b], lens[b] + n, device="cuda")
        pg, off = table[b].long()[slot // page], slot % page
        for name, x, w, out in (("q", was, weights[0], got[rows]), ("k", k, weights[1], k_cache[pg, off])):
            if positions is None:
                want, size = tree.append(x[rows], slot, w, 1e-5, freq, interleaved, scale)
            else:  # an axis at a time: its pairs alone turn
                want, size = tree.append(x[rows], slot, w, 1e-5, None, interleaved, scale)
                for axis in range(axes):
                    one, s = tree.append(x[rows], positions[axis, rows], w, 1e-5, freq, interleaved, scale)
                    for j in torch.nonzero(axis_of == axis).flatten().tolist():
                        for d in ((2 * j, 2 * j + 1) if interleaved else (j, j + half)):
                            want[..., d], size[..., d] = one[..., d], s[..., d]
            close(out, want, tree.append_tolerance(want, size, dtype), f"{name} of request {b}")
        assert torch.equal(v_cache[pg, off], v[rows])
        used_k[pg, off], used_v[pg, off] = k_cache[pg, off], v_cache[pg, off]
    same = lambda a, b: torch.equal(a.view(torch.int16), b.view(torch.int16))  # noqa: E731
    assert same(k_cache.contiguous(), used_k.contiguous()) and same(v_cache.contiguous(), used_v.contiguous())
    assert torch.equal(got[int(cu[-1]):], was[int(cu[-1]):] if in_place else torch.full_like(was[int(cu[-1]):], 7.0))


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("new,lens,Hq,Hkv,D,page,axes,rot,interleaved,norm,scale", [
    ([1], [0], 1, 1, 8, 16, 0, 8, False, True, 1.0),
    ([1], [1999], 32, 8, 128, 16, 3, 128, False, True, 1.0),
    ([517], [0], 32, 8, 128, 16, 0, 128, False, True, 1.0),
    ([30, 0, 1, 200], [100, 7, 0, 33], 8, 2, 128, 64, 3, 128, False, True, 1.0),
    ([30, 5], [100, 7], 8, 2, 128, 64, 3, 64, True, False, 0.7),
    ([70], [3], 7, 1, 80, 24, 2, 40, False, True, 1.0),      # halves that do not begin at a piece
    ([70], [3], 5, 5, 96, 1, 4, 36, False, True, 1.0),
    ([9, 140], [5, 140], 9, 3, 64, 3, 0, 0, False, True, 1.0),
    ([9, 140], [5, 140], 9, 3, 64, 3, 2, 0, True, False, 1.0),  # a copy
    ([33], [10], 3, 3, 40, 8, 1, 40, True, True, 1.2),
    ([4000, 1, 2500], [0, 50, 100], 4, 1, 64, 128, 3, 64, False, True, 1.0),
    ([11], [2], 1, 1, 120, 100, 2, 120, False, True, 1.0),
])
def test_append(sv, dtype, new, lens, Hq, Hkv, D, page, axes, rot, interleaved, norm, scale):  # noqa: F811
    run_append(sv, 3, new, lens, Hq, Hkv, D, page, dtype, axes=axes, rot=rot, interleaved=interleaved, norm=norm,
               scale=scale, spare=3 * (len(new) - 1))


@pytest.mark.parametrize("layout", ["heads", "pairs"])
def test_append_layouts_and_in_place(sv, layout):  # noqa: F811
    run_append(sv, 5, [40, 3], [90, 10], 8, 2, 64, 16, BF16, axes=2, rot=64, interleaved=False, norm=True,
               scale=1.0, layout=layout, spare=2, in_place=True)


def test_append_many_requests_and_far_positions(sv):  # noqa: F811
    rng = np.random.default_rng(1)
    new, lens = [int(x) for x in rng.integers(0, 4, 1200)], [int(x) for x in rng.integers(0, 60, 1200)]
    run_append(sv, 7, new, lens, 2, 1, 64, 16, F16, axes=3, rot=64, interleaved=False, norm=False, scale=1.0,
               far=10 ** 9)


def test_append_one_axis_as_a_row(sv):  # noqa: F811
    """positions [T] is one axis; the slots themselves give what no positions give, as append_nodes does."""
    gen = torch.Generator(device="cuda").manual_seed(9)
    q, k, v = (torch.randn(20, h, 64, generator=gen, device="cuda").to(BF16) for h in (4, 2, 2))
    freq = 10000.0 ** (-torch.arange(32, device="cuda") / 32)
    made = []
    for how in ("slots", "row", "nodes"):
        kc, vc = (torch.zeros(4, 16, 2, 64, dtype=BF16, device="cuda") for _ in "kv")
        table = i32([[2, 0, 1, 3]])
        if how == "nodes":
            out, _ = sv.append_nodes(q[None], k[None], v[None], kc, vc, table, i32([30]), freq)
            out = out[0]
        else:
            at = torch.arange(30, 50, device="cuda", dtype=torch.int32) if how == "row" else None
            out, _ = sv.append_chunk(q, k, v, kc, vc, table, i32([30]), i32([0, 20]), freq, positions=at)
        made.append((out, kc, vc))
    for other in made[1:]:
        assert all(torch.equal(a, b) for a, b in zip(made[0], other))


def test_append_flags_bad_requests(sv):  # noqa: F811
    new, lens = [20, 30, 9], [100, 40, 7]
    cu = np.concatenate([[0], np.cumsum(new)])
    gen = torch.Generator(device="cuda").manual_seed(11)
    q, k, v = (torch.randn(59, h, 64, generator=gen, device="cuda").to(BF16) for h in (4, 2, 2))
    freq = 10000.0 ** (-torch.arange(32, device="cuda") / 32)
    table = torch.randperm(30, generator=gen, device="cuda")[:24].view(3, 8).to(torch.int32)

    def call(lens=lens, cu=cu, table=table, **kw):
        kc, vc = (torch.full((30, 16, 2, 64), 3.0, dtype=BF16, device="cuda") for _ in "kv")
        out = torch.full_like(q, 7.0)
        _, status = sv.append_chunk(q, k, v, kc, vc, table, i32(lens), i32(cu), freq, q_out=out, **kw)
        return out, kc, vc, status.tolist()

    want = call()
    assert want[3] == [0, 0, 0]

    def pages(c, b):
        return c[table[b].long()]

    for kw, flag in [(dict(lens=[100, -1, 7]), sv.DEV_BAD_CACHE), (dict(lens=[100, 99, 7]), sv.DEV_BAD_CACHE),
                     (dict(table=torch.where(table == table[1, 4], 30, table)), sv.DEV_BAD_CACHE),
                     (dict(table=torch.where(table == table[1, 2], -1, table)), sv.DEV_BAD_CACHE)]:
        out, kc, vc, status = call(**kw)
        assert status == [0, flag, 0]
        assert (out[20:50] == 0).all() and torch.equal(out[:20], want[0][:20]) and torch.equal(out[50:], want[0][50:])
        assert (pages(kc, 1) == 3.0).all() and (pages(vc, 1) == 3.0).all()
        for b in (0, 2):
            assert torch.equal(pages(kc, b), pages(want[1], b)) and torch.equal(pages(vc, b), pages(want[2], b))
    # a page that the chunk does not write need not exist
    out, kc, vc, status = call(table=torch.where(table == table[1, 0], -7, table))
    assert status == [0, 0, 0] and torch.equal(out, want[0])
    # cu_tokens that falls or leaves the rows
    out, kc, vc, status = call(cu=[0, 20, 10 ** 6, 59])
    assert status == [0, sv.DEV_BAD_DRAFT_LEN, sv.DEV_BAD_DRAFT_LEN]
    assert torch.equal(out[:20], want[0][:20]) and (out[20:] == 7.0).all()
    assert (pages(kc, 1) == 3.0).all() and (pages(kc, 2) == 3.0).all()
    out, kc, vc, status = call(cu=[0, 20, 10, 10])
    assert status == [0, sv.DEV_BAD_DRAFT_LEN, 0]
    assert torch.equal(out[:20], want[0][:20]) and (out[20:] == 7.0).all()
    # an axis that is none: every request
    at = torch.zeros(2, 59, dtype=torch.int32, device="cuda")
    for axis in (-1, 2):
        of = torch.zeros(32, dtype=torch.int32, device="cuda")
        of[31] = axis
        out, kc, vc, status = call(positions=at, axis_of=of)
        assert status == [sv.DEV_BAD_POSITION] * 3 and (out == 0).all() and (kc == 3.0).all()


def test_append_no_tokens(sv):  # noqa: F811
    kc, vc = (torch.full((4, 16, 2, 64), 3.0, dtype=BF16, device="cuda") for _ in "kv")
    q, k = (torch.zeros(0, h, 64, dtype=BF16, device="cuda") for h in (4, 2))
    freq = torch.ones(32, device="cuda")
    for at, of in [(None, None), (torch.zeros(3, 0, dtype=torch.int32, device="cuda"), i32(np.zeros(32)))]:
        out, status = sv.append_chunk(q, k, k, kc, vc, i32([[0, 1], [2, 3]]), i32([4, 5]), i32([0, 0, 0]), freq,
                                      positions=at, axis_of=of)
        assert out.shape == (0, 4, 64) and status.tolist() == [0, 0] and (kc == 3.0).all()


def test_append_on_another_stream_and_in_a_graph(sv):  # noqa: F811
    gen = torch.Generator(device="cuda").manual_seed(13)
    q, k, v = (torch.randn(50, h, 64, generator=gen, device="cuda").to(BF16) for h in (4, 2, 2))
    freq = 10000.0 ** (-torch.arange(32, device="cuda") / 32)
    kc, vc = (torch.zeros(10, 16, 2, 64, dtype=BF16, device="cuda") for _ in "kv")
    table, lens, cu = i32(np.arange(10).reshape(2, 5)), i32([3, 20]), i32([0, 10, 50])
    call = lambda **kw: sv.append_chunk(q, k, v, kc, vc, table, lens, cu, freq, **kw)  # noqa: E731
    want = call()[0]
    cache = kc.clone(), vc.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    kc.zero_(), vc.zero_()
    torch.cuda.synchronize()
    got, _ = call(stream=side)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(kc, cache[0]) and torch.equal(vc, cache[1])
    out, status = torch.zeros_like(q), i32([9, 9])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(q_out=out, status=status)
    kc.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(kc, cache[0]) and status.tolist() == [0, 0]


# ----------------------------------------------------------------- all of them


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_a_prompt_in_chunks_then_a_drafted_chain(sv, dtype):  # noqa: F811
    """A prompt of positions on three axes goes in by chunks, beside a second request; then a chain is
    drafted and verified on the same cache by the tree's operators.  Every output against its plain form."""
    gen = torch.Generator(device="cuda").manual_seed(17)
    Hq, Hkv, D, page, half = 8, 2, 64, 16, 32
    freq = 10000.0 ** (-torch.arange(half, device="cuda") / half)
    axis_of = i32(np.arange(half) % 3)
    kc, vc = (torch.full((60, page, Hkv, D), float("nan"), dtype=dtype, device="cuda") for _ in "kv")
    table = torch.randperm(60, generator=gen, device="cuda")[:56].view(2, 28).to(torch.int32)
    lens = [0, 0]
    for new in ([100, 1], [150, 200], [1, 33]):
        T, cu = sum(new), np.concatenate([[0], np.cumsum(new)])
        qkv = torch.randn(T, (Hq + 2 * Hkv) * D, generator=gen, device="cuda").to(dtype)
        q, k, v = (x.unflatten(-1, (-1, D)) for x in qkv.split([Hq * D, Hkv * D, Hkv * D], -1))
        pos = torch.randint(0, 5000, (3, T), generator=gen, device="cuda", dtype=torch.int32)
        rotated, status = sv.append_chunk(q, k, v, kc, vc, table, i32(lens), i32(cu), freq, positions=pos,
                                          axis_of=axis_of)
        assert status.tolist() == [0, 0]
        out, status = sv.chunk_attention(rotated, kc, vc, table, i32(lens), i32(cu), cap=30.0, window=160,
                                         prefix_lens=i32([4, 4]), longest=max(new))
        assert status.tolist() == [0, 0]
        want, tol = ref.attention(rotated, kc, vc, table, lens, cu, D ** -0.5, 30.0, 160, [4, 4])
        close(out, want, tol)
        lens = [a + b for a, b in zip(lens, new)]
    nodes = torch.randn(2, 5, (Hq + 2 * Hkv) * D, generator=gen, device="cuda").to(dtype)
    q, k, v = (x.unflatten(-1, (-1, D)) for x in nodes.split([Hq * D, Hkv * D, Hkv * D], -1))
    rotated, status = sv.append_nodes(q, k, v, kc, vc, table, i32(lens), freq)
    assert status.tolist() == [0, 0]
    out, status = sv.tree_attention(rotated, kc, vc, table, i32(lens))
    assert status.tolist() == [0, 0]
    # a chain is a chunk: both attentions over the same cache
    want, tol = ref.attention(rotated.flatten(0, 1), kc, vc, table, lens, [0, 5, 10], D ** -0.5)
    close(out.flatten(0, 1), want, tol)
    chunk, _ = sv.chunk_attention(rotated.flatten(0, 1), kc, vc, table, i32(lens), i32([0, 5, 10]))
    close(chunk, want, tol)
