"""Beam selection and reordering against plain 64-bit forms, and a tree drafted
with them level by level."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import prompt_reference as ref  # noqa: E402
from test_gpu_tree import BF16, F16, F32, f32, i32, sv  # noqa: E402, F401

pytestmark = pytest.mark.gpu


def check(sv, z, scores, K, ended=None, end_token=0, **kw):  # noqa: F811
    """Against the reference.  A score is its row's sum of exponentials (each within 2^-22 and the
    argument's rounding, 2^-23 of it: off by at most 2^-20 for arguments that matter), differences in
    64 bits and one rounding.  Candidates of two rows that are nearer than both rows' sums are known may
    change places, so a place has either the reference's candidate or one whose score in the
    reference is within 2^-19 of it; none twice, and of one row in its order."""
    got = sv.select_beams(z, f32(scores), K, ended=None if ended is None else i32(ended), end_token=end_token, **kw)
    torch.cuda.synchronize()
    out, tokens, beams, flags = (x.cpu().numpy() for x in got)
    assert flags.tolist() == [0] * len(scores)
    want, names, rows, all_rows = ref.select(z.float().cpu().numpy(), np.asarray(scores, np.float32), K, ended,
                                             end_token)
    live = np.isfinite(want)
    assert np.array_equal(out == -np.inf, ~live)
    assert (np.abs(out[live] - want[live]) <= np.abs(want[live]) * 2.0 ** -23 + 2.0 ** -20).all()
    other = (tokens != names) | (beams != rows)
    for b, k in zip(*np.nonzero(other)):
        assert abs(all_rows[b][beams[b, k]][tokens[b, k]] - want[b, k]) <= 2.0 ** -19, (b, k)
    for b in np.nonzero(other.any(1))[0]:
        for w in range(z.shape[1]):
            mine, theirs = tokens[b][beams[b] == w], names[b][rows[b] == w]
            n = min(len(mine), len(theirs))
            assert np.array_equal(mine[:n], theirs[:n]), (b, w)
    return got


def normal(seed, *shape, dtype=F32, scale=3.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (scale * torch.randn(*shape, generator=gen, device="cuda")).to(dtype)


def totals(seed, B, W):
    return -np.random.default_rng(seed).exponential(4.0, (B, W)).astype(np.float32)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,W,K,V", [
    (1, 1, 1, 1), (1, 1, 5, 3), (2, 3, 3, 7), (3, 1, 8, 1000), (2, 8, 8, 8192), (2, 8, 8, 8193), (1, 4, 64, 16385),
    (2, 64, 64, 2050), (5, 7, 13, 32003), (1, 8, 8, 128256), (3, 5, 33, 50001), (200, 2, 3, 501), (1, 64, 1, 9000),
    (1, 2, 17, 524288),
])
def test_select(sv, dtype, B, W, K, V):  # noqa: F811
    z = normal(B + 7 * W + K, B, W, V, dtype=dtype)
    check(sv, z, totals(K, B, W), K)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_select_beams_ended_and_not_in_play(sv, dtype):  # noqa: F811
    rng = np.random.default_rng(3)
    z, scores = normal(3, 6, 5, 3001, dtype=dtype), totals(3, 6, 5)
    ended = rng.integers(0, 2, (6, 5))
    ended[1] = 1                # fewer candidates than places
    scores[2, 1:] = -np.inf     # a first step: one beam in play
    scores[3] = -np.inf         # none
    ended[4] = 0
    z[4, 2:] = float("-inf")    # rows in which nothing is allowed
    z[2, 1:] = float("nan")     # of beams not in play: not read
    check(sv, z, scores, 7, ended * np.where(scores > -np.inf, 5, -3), end_token=2)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_select_few_allowed(sv, dtype):  # noqa: F811
    """A grammar leaves few tokens, or fewer than places; the lowest finite values are candidates."""
    z = torch.full((3, 2, 20000), float("-inf"), dtype=dtype, device="cuda")
    z[0, 0, 19999], z[0, 1, 3], z[0, 1, 8191] = 1.0, 2.0, -1.0
    z[1, 0, ::97] = normal(5, 207, dtype=dtype)
    z[2, 0] = normal(6, 20000, dtype=dtype)
    z[2, 1, 8192:8300] = -3e38
    z[2, 1, 5] = -3.3e38
    check(sv, z, [[-1.0, -2.5], [-0.5, -np.inf], [-700.0, -0.125]], 40)


def test_select_scores_below_the_lowest(sv):  # noqa: F811
    """A score that rounds to -inf is no candidate: no place has -inf and a token."""
    low = torch.finfo(F32).min
    z = torch.full((2, 2, 5), low, device="cuda")
    z[:, :, 3] = 1.0
    out, tokens, beams, status = sv.select_beams(z, f32([[low, -1.0], [low, low]]), 10)
    assert status.tolist() == [0, 0]
    # request 0: beam 1's token 3; beam 0's and beam 1's masked ones, alike in 64 bits; beam 0's masked
    # ones are 2 low
    assert tokens[0].tolist() == [3, 3, 0, 1, 2, 4, -1, -1, -1, -1]
    assert beams[0].tolist() == [1, 0, 1, 1, 1, 1, -1, -1, -1, -1]
    assert out[0].tolist() == [-1.0] + [low] * 5 + [float("-inf")] * 4
    assert tokens[1].tolist() == [3, 3] + [-1] * 8 and beams[1].tolist() == [0, 1] + [-1] * 8


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("far", [-1e9, -1e30, -3.4028234663852886e38, 1e30])
def test_select_far_scores_keep_the_order_of_logits(sv, dtype, far):  # noqa: F811
    """Beams put out of the others' way by a large score: a beam's own tokens are still in the order of
    its logits, and its ties in that of the tokens."""
    for V, K, B in ((40, 32, 2), (9000, 64, 300)):  # (with few candidates, and one after the other)
        z = normal(37, B, 2, V, dtype=dtype)
        out, tokens, beams, status = sv.select_beams(z, f32([[far, -float("inf")], [-float("inf"), far]] * (B // 2)), K)
        assert (status == 0).all()
        for b in (0, 1, B - 1):
            row = z[b, b % 2].float().cpu().numpy()
            assert tokens[b].tolist() == np.lexsort((np.arange(V), -row))[:K].tolist()
            assert (beams[b] == b % 2).all()
    z = torch.zeros(1, 64, 64, device="cuda", dtype=dtype)  # more alike than are sorted at once
    z[:, :, 1::2] = torch.arange(32, device="cuda", dtype=dtype)
    tokens, beams = sv.select_beams(z, f32([[far] * 64]), 64)[1:3]
    want = list(range(63, 0, -2)) + list(range(0, 64, 2))
    if far != -1e9:  # (there the sums of 64 rows tell the logits apart)
        assert beams[0].tolist() == [0] * 64 and sorted(tokens[0].tolist()) == list(range(64))
        order = tokens[0].tolist()
        assert order == [t for t in want if t != 1 and t % 2] + sorted(t for t in want if t == 1 or t % 2 == 0)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_select_more_candidates_than_are_kept(sv, dtype):  # noqa: F811
    """64 beams' lists of 64 in three parts or more: what a block's shared memory does not hold is read again."""
    check(sv, normal(41, 1, 64, 20000, dtype=dtype), totals(41, 1, 64), 64)


def test_select_ties_go_to_the_lowest(sv):  # noqa: F811
    """Equal scores: the lower beam, then the lower token, however many there are."""
    for V in (50, 8192, 40003):
        z = torch.zeros(2, 3, V, device="cuda", dtype=BF16)
        z[1, :, V // 2:] = 1.0
        z[1, 1, 7] = 1.0
        out, tokens, beams, status = sv.select_beams(z, f32([[-1.0, -1.0, -1.0], [-2.0, -1.0, -2.0]]), 20)
        assert status.tolist() == [0, 0]
        assert tokens[0].tolist() == list(range(20)) and beams[0].tolist() == [0] * 20
        assert tokens[1].tolist() == [7] + list(range(V // 2, V // 2 + 19)) and beams[1].tolist() == [1] * 20
        assert (out[0] == out[0, 0]).all()
    # 0 and -0 are equal; so are all rows' entries past the first tile
    z = torch.full((1, 1, 30000), -4.0, device="cuda")
    z[0, 0, 100], z[0, 0, 20000], z[0, 0, 29999] = -0.0, 0.0, 0.0
    assert sv.select_beams(z, f32([[0.0]]), 4)[1].tolist() == [[100, 20000, 29999, 0]]


def test_select_rising_and_falling_rows(sv):  # noqa: F811
    """Every tile has K better entries than the ones before, or none."""
    up = torch.arange(50000, device="cuda", dtype=F32) * 0.01
    z = torch.stack([up, up.flip(0), up * 1.5])[None].contiguous()
    check(sv, z, [[-1.0, -1.5, -3.0]], 64)
    one = torch.full((1, 2, 9000), -50.0, device="cuda")
    one[0, 0, 8999], one[0, 1, 0] = 50.0, 60.0
    check(sv, one + normal(1, 1, 2, 9000, scale=0.1), [[-1.0, -1.5]], 8)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_select_strides_and_alignments(sv, dtype):  # noqa: F811
    B, W, V = 2, 3, 10007
    wide = normal(11, B, W + 1, V + 24, dtype=dtype)
    for first in range(9):  # rows that begin anywhere
        check(sv, wide[:, 1:, first:first + V], totals(11, B, W), 6)
    check(sv, wide[:1, :, :V].expand(2, W + 1, V), totals(12, 2, W + 1), 6)
    flat = normal(13, 1, 1, V, dtype=dtype).expand(2, 3, V)  # one row for all
    check(sv, flat, [[-1.0, -1.5, -2.25], [-3.0, -0.5, -0.75]], 4)


def test_select_flags_bad_requests(sv):  # noqa: F811
    z, scores = normal(17, 6, 2, 9001), totals(17, 6, 2)
    z[1, 1, 9000] = float("nan")
    z[2, 0, 5] = float("inf")
    z[3, 1] = float("nan")
    scores[4, 0] = np.nan
    scores[5, 1] = np.inf
    out, tokens, beams, status = sv.select_beams(z, f32(scores), 4)
    bad = [0] + [sv.DEV_BAD_ROW] * 3 + [sv.DEV_BAD_BEAM] * 2
    assert status.tolist() == bad
    assert (out[1:] == float("-inf")).all() and (tokens[1:] == -1).all() and (beams[1:] == -1).all()
    check(sv, z[:1], scores[:1], 4)


def test_select_the_same_every_time_and_in_graphs(sv):  # noqa: F811
    z, scores = normal(19, 8, 8, 50000, dtype=BF16), f32(totals(19, 8, 8))
    want = sv.select_beams(z, scores, 16)
    for fill in (0, 255):
        ws = sv.BeamWorkspace(8, 8, 16, 50000, device="cuda")
        ws.tensor.fill_(fill)
        again = sv.select_beams(z, scores, 16, workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(want, again))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = sv.select_beams(z, scores, 16, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    outs = [torch.zeros_like(x) for x in want]
    graphs = []
    for _ in range(2):  # two graphs that take turns on one workspace
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            sv.select_beams(z, scores, 16, workspace=ws, out_scores=outs[0], tokens=outs[1], beams=outs[2],
                            status=outs[3])
        graphs.append(g)
    for g in graphs + graphs:
        for o in outs:
            o.fill_(9)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, outs))


def test_select_a_workspace_for_the_largest_batch(sv):  # noqa: F811
    ws = sv.BeamWorkspace(64, 8, 8, 32003, device="cuda")
    for B, W, K, V in ((64, 8, 8, 32003), (56, 8, 8, 32003), (40, 8, 8, 30000), (13, 8, 8, 32003), (1, 8, 8, 32003),
                       (11, 3, 8, 20000), (33, 8, 1, 16385)):
        for dtype in (BF16, F32):
            check(sv, normal(B, B, W, V, dtype=dtype), totals(B, B, W), K, workspace=ws)


@pytest.mark.parametrize("dtype,V,low,every", [(F32, 1 << 19, -1.1171624660491943, 4), (BF16, 1 << 20, -0.83984375, 8)])
def test_select_long_rows_sums(sv, dtype, V, low, every):  # noqa: F811
    """Rows of so many requests that a block has a whole one: a lane adds the same sum 128 times, of a size that
    one 32-bit number would round the same way each time, 1.9e-6 of the sum in the end.  Of the
    sum the exponentials are off by 2^-22 and the argument's rounding, 2^-24 of at most 1.7, and those of a
    step by 10 roundings: 2^-20 of it, and as much of its logarithm."""
    row = torch.full((V,), low, dtype=dtype, device="cuda")
    row[::every] = 0.0
    z = row.expand(8, 64, V)
    out, tokens, beams, status = sv.select_beams(z, f32([[12.5] * 64] * 8), 1)
    assert (status == 0).all() and (tokens == 0).all() and (beams == 0).all()
    want = 12.5 - np.log(V // every * (1.0 + (every - 1) * np.exp(np.float64(low))))
    assert abs(want) < 1.0 and np.abs(out.cpu().double().numpy() - want).max() <= 2.0 ** -20


def test_select_offsets_past_32_bits(sv):  # noqa: F811
    z = normal(23, 3, 2, 1000, dtype=BF16)
    far = torch.empty(2 ** 32 + 2000, dtype=BF16, device="cuda").as_strided((3, 2, 1000), (2 ** 31, 1000, 1))
    far.copy_(z)
    check(sv, far, totals(23, 3, 2), 5)


def test_select_refusals(sv):  # noqa: F811
    z, scores = normal(29, 2, 3, 100), f32(totals(29, 2, 3))
    for kw in (dict(status=i32([0])), dict(beams=i32(np.zeros((2, 4)))), dict(tokens=torch.zeros(2, 3, device="cuda")),
               dict(out_scores=torch.zeros(2, 1, device="cuda").expand(2, 3))):
        with pytest.raises(ValueError):
            sv.select_beams(z, scores, 3, **kw)
    with pytest.raises(ValueError):
        sv.select_beams(z, scores, 65)
    with pytest.raises(sv.SpecVerifyError):  # 2 x 3 lists of 64 do not fit where one of 1 does
        sv.select_beams(z, scores, 64, workspace=sv.BeamWorkspace(1, 1, 1, 100, device="cuda"))


# -------------------------------------------------------------------- reorder


def moved(beams, x, out):
    """What out becomes."""
    out = out.clone()
    for b, row in enumerate(beams.tolist()):
        for k, w in enumerate(row):
            if w >= 0:
                out[b, k] = x[b, w]
    return out


@pytest.mark.parametrize("B,W,K", [(1, 1, 1), (2, 3, 5), (3, 8, 8), (2, 16, 16), (2, 17, 9), (2, 30, 32), (1, 64, 64),
                                   (70, 4, 2)])
def test_reorder(sv, B, W, K):  # noqa: F811
    rng = np.random.default_rng(B + W + K)
    gen = torch.Generator(device="cuda").manual_seed(W)
    beams = i32(rng.integers(-1, W, (B, K)))
    states = [normal(1, B, W, 4096, dtype=BF16), normal(2, B, W, 3, 5), normal(3, B, W, 1, dtype=F16),
              torch.randint(0, 9, (B, W, 77), generator=gen, device="cuda", dtype=torch.uint8),
              torch.randint(0, 9, (B, W, 1001), generator=gen, device="cuda", dtype=torch.int32),
              torch.randint(0, 9, (B, W), generator=gen, device="cuda") > 4,
              normal(4, B, W, 7, dtype=torch.float64), normal(5, B, W, 0), normal(6, B, W, 2050, dtype=F16)[..., 1:]]
    outs = [torch.full((B, K, *x.shape[2:]), 1, dtype=x.dtype, device="cuda") for x in states]
    want = [moved(beams, x, o) for x, o in zip(states, outs)]
    got, status = sv.reorder_beams(beams, states, out=outs)
    torch.cuda.synchronize()
    assert status.tolist() == [0] * B
    assert all(a is b for a, b in zip(got, outs)) and all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("W", [1, 2, 8, 13, 32, 64])
def test_reorder_in_place(sv, W):  # noqa: F811
    """Every old state is read before it is overwritten, whatever goes where."""
    rng = np.random.default_rng(W)
    rows = [np.arange(W), np.arange(W)[::-1], np.roll(np.arange(W), 1), np.zeros(W), rng.integers(-1, W, W),
            rng.permutation(W), np.full(W, -1)]
    beams = i32(np.stack(rows))
    for x in (normal(W, 7, W, 2055, dtype=BF16), normal(W, 7, W, 515),
              normal(W, 7, W, 640, dtype=F16), normal(W, W, 7, 33).transpose(0, 1)):
        want = moved(beams, x, x)
        got, status = sv.reorder_beams(beams, x)
        torch.cuda.synchronize()
        assert got is x and status.tolist() == [0] * 7 and torch.equal(x, want)


def test_reorder_flags_bad_requests(sv):  # noqa: F811
    x = normal(1, 3, 4, 100)
    out = torch.full((3, 2, 100), 7.0, device="cuda")
    beams = i32([[0, 3], [4, 0], [-2, 1]])
    _, status = sv.reorder_beams(beams, x, out=out)
    assert status.tolist() == [0, sv.DEV_BAD_BEAM, sv.DEV_BAD_BEAM]
    assert torch.equal(out[0], x[0, [0, 3]]) and (out[1:] == 7.0).all()


def test_reorder_many_requests(sv):  # noqa: F811
    """More requests than one axis of a grid has here: none behind the last is looked at."""
    B = 32768 + 5
    rng = np.random.default_rng(2)
    beams = rng.integers(-1, 3, (B, 2))
    x = normal(7, B, 3, 5)
    out = torch.zeros(B, 2, 5, device="cuda")
    status = torch.full((B + 64,), 9, dtype=torch.int32, device="cuda")
    _, flags = sv.reorder_beams(i32(beams), x, out=out, status=status[:B])
    torch.cuda.synchronize()
    at = torch.as_tensor(beams).cuda()
    want = torch.where(at[:, :, None] >= 0, x.gather(1, at.clamp(min=0)[:, :, None].expand(B, 2, 5)), 0.0)
    assert torch.equal(out, want) and (flags == 0).all() and (status[B:] == 9).all()


def test_select_many_requests(sv):  # noqa: F811
    z, scores = normal(31, 5000, 2, 33, dtype=BF16), totals(31, 5000, 2)
    check(sv, z, scores, 3)


def test_reorder_strides_streams_and_graphs(sv):  # noqa: F811
    layers = normal(3, 4, 3, 5, 64, dtype=BF16)  # [layers, B, W, ...]: a state to each
    beams = i32([[1, 1, 0, 4, 2], [4, 3, 2, 1, 0], [-1, 0, 0, 0, 0]])
    outs = torch.zeros_like(layers)
    want = torch.stack([moved(beams, x, o) for x, o in zip(layers, outs)])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    sv.reorder_beams(beams, list(layers), out=list(outs), stream=side)
    side.synchronize()
    assert torch.equal(outs, want)
    status = i32([5, 5, 5])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.reorder_beams(beams, list(layers), out=list(outs), status=status)
    outs.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs, want) and status.tolist() == [0, 0, 0]
    far = torch.empty(2 ** 32 + 4096, dtype=torch.uint8, device="cuda").as_strided((3, 5, 16), (2 ** 31, 64, 1))
    far.copy_(torch.arange(240, device="cuda").view(3, 5, 16))
    got, _ = sv.reorder_beams(beams, far, out=torch.zeros(3, 5, 16, dtype=torch.uint8, device="cuda"))
    assert torch.equal(got, moved(beams, far, torch.zeros_like(got)))


def test_reorder_refusals(sv):  # noqa: F811
    x, beams = normal(1, 2, 3, 8), i32([[0, 1, 2], [0, 0, 0]])
    with pytest.raises(ValueError):
        sv.reorder_beams(beams, x, status=i32([0]))
    with pytest.raises(sv.SpecVerifyError):
        sv.reorder_beams(beams, [x] * 33, out=[torch.zeros_like(x) for _ in range(33)])


def test_reorder_states_of_one_tensor(sv):  # noqa: F811
    """Views that lie between one another's beams are moved beside one another; places that two would write, or one
    write and the other read, are refused, as blocks of a call run in any order."""
    beams = i32([[2, 0, 1], [1, 1, 2]])
    whole = normal(7, 2, 3, 4, 16)
    want = moved(beams, whole, whole)
    views = [whole[:, :, i] for i in range(4)]
    sv.reorder_beams(beams, views)
    assert torch.equal(whole, want)
    wide = normal(8, 2, 6, 16)
    want = moved(beams, wide[:, :3], wide[:, 3:])
    sv.reorder_beams(beams, wide[:, :3], out=wide[:, 3:])
    assert torch.equal(wide[:, 3:], want)
    turned = normal(9, 3, 2, 16).transpose(0, 1)  # a beam's requests beside one another
    want = moved(beams, turned, turned)
    sv.reorder_beams(beams, turned)
    assert torch.equal(turned, want)
    x, y = normal(10, 2, 3, 16), normal(11, 2, 3, 16)
    was = x.clone(), y.clone(), wide.clone(), whole.clone()
    for states, out in [((x, x), None), ((x, x[:, :, :8]), None), ((x, y), (y, x)), ((x, y), (torch.zeros_like(x), x)),
                        ((x, y), (y, torch.zeros_like(x))), ((whole[:, :, 0:2], whole[:, :, 1:3]), None),
                        ((wide[:, :3],), (wide[:, 2:5],)), ((wide[:, :3],), (wide[:, 1:4],)),
                        ((wide[:, 3:],), (wide[:, 1:4],)), ((x[:, :, 4:8], x[:, :, 7:11]), None)]:
        with pytest.raises(sv.SpecVerifyError):
            sv.reorder_beams(beams, states, out=out)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(was, (x, y, wide, whole)))


# --------------------------------------------------------- a tree, level by level


def test_a_tree_is_drafted_and_verified(sv):  # noqa: F811
    """Three levels of four nodes: the best of the last level's continuations, their features and
    texts moved along; then the tree's greedy verification finds the path that the target says."""
    B, W, V, levels = 2, 4, 700, 3
    N = 1 + levels * W
    gen = torch.Generator(device="cuda").manual_seed(5)
    head = torch.randn(V, 32, generator=gen, device="cuda")
    embed = torch.randn(V, 32, generator=gen, device="cuda")
    features = torch.randn(B, 1, 32, generator=gen, device="cuda")
    scores = torch.zeros(B, 1, device="cuda")
    nodes = torch.zeros(B, 1, dtype=torch.int32, device="cuda")  # the beams' node numbers
    tokens, parents = i32(np.zeros((B, N))), i32(np.full((B, N), -1))
    texts = torch.full((B, 1, levels), -1, dtype=torch.int32, device="cuda")
    plain = [[(0.0, [], features[b, 0].double())] for b in range(B)]
    for level in range(levels):
        scores, token, beam, status = sv.select_beams(features @ head.T, scores, W)
        assert status.tolist() == [0] * B
        K = token.shape[1]
        out = [torch.zeros(B, K, *x.shape[2:], dtype=x.dtype, device="cuda") for x in (features, texts, nodes)]
        (features, texts, up), status = sv.reorder_beams(beam, (features, texts, nodes), out=out)
        assert status.tolist() == [0] * B
        texts[:, :, level] = token
        features = 0.5 * features + embed[token.long()]
        first = 1 + level * W
        nodes = torch.arange(first, first + W, device="cuda", dtype=torch.int32).expand(B, W).contiguous()
        tokens[:, first:first + W], parents[:, first:first + W] = token, up
        for b in range(B):
            pool = []
            for total, text, f in plain[b]:
                z = head.double() @ f
                for v, x in enumerate((total + torch.log_softmax(z, 0)).tolist()):
                    pool.append((x, text + [v], f))
            pool.sort(key=lambda c: -c[0])
            plain[b] = [(x, text, 0.5 * f + embed[text[-1]].double()) for x, text, f in pool[:W]]
            assert texts[b, :, :level + 1].tolist() == [text for _, text, _ in plain[b]]
            assert np.allclose(scores[b].tolist(), [x for x, _, _ in plain[b]], rtol=0, atol=1e-3)
    # a target that says the second drafted text of each request
    target = torch.zeros(B, N, V, device="cuda")
    for b in range(B):
        at, said = 0, texts[b, 1].tolist()
        for depth, want in enumerate(said + [9]):
            target[b, at, want] = 5.0
            if depth < levels:
                first = 1 + depth * W
                at = next(i for i in range(first, first + W)
                          if int(parents[b, i]) == at and int(tokens[b, i]) == want)
    accepted, said, _ = sv.verify_tree_greedy(target, parents, tokens, i32([N, N]))[:3]
    assert accepted.tolist() == [levels] * B
    for b in range(B):
        assert said[b, :levels + 1].tolist() == texts[b, 1].tolist() + [9]
