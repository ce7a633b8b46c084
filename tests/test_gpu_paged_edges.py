"""The paged operators where several tiles of a sequence meet in one warp: bases and units that move, stages that
are used again, pages that are not there, scales at the ends of their range. Against the definitions in 64 bits."""
import numpy as np
import pytest

from test_gpu_paged_ops import B, Paged, rotate_ref, rotation_tol, stream  # noqa: F401  (B: the fixture)

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def call(a):
    a.call()
    a.B.op_sync(stream())
    return a.out.double().cpu().numpy()


def positive_values(a):
    """Values of one sign, so that an output is as large as they are and a part of the sum that is lost shows."""
    for s, x in enumerate(a.c.rows):
        y = x.copy()
        y[1] = np.abs(y[1])
        a.c.rows[s] = a.c._put(s, y)


def scale_rows(a, s, plane, rows, factor):
    """Multiplies the scales (e4m3 pages) of some rows of a sequence, as fp32 holds the products."""
    c = a.c
    pid, off = c.places(s, c.rows[s].shape[1])
    p, o = (torch.from_numpy(t[rows].astype(np.int64)).cuda() for t in (pid, off))
    f = torch.from_numpy(np.broadcast_to(np.asarray(factor, np.float64), len(rows)).copy()).cuda()[:, None]
    old = c.scales[plane][p, :, o].double()
    new = (old * f).float()
    c.scales[plane][p, :, o] = new
    c.rows[s][plane][rows] *= (new.double() / old).cpu().numpy()[..., None]


def drop_pages(a, s, cols):
    """Page ids outside the pool: those pages' rows are zeros."""
    bad = [-1, a.c.n_pages, 2 ** 31 - 1, -2 ** 31]
    for i, col in enumerate(cols):
        a.c.d_table[s, int(col)] = bad[i % 4]
        a.c.rows[s][:, int(col) * a.c.page:(int(col) + 1) * a.c.page] = 0


# ---- batches with empty sequences ------------------------------------------------------------
def test_many_prompts_then_empty_ones(B):  # noqa: F811
    """1024 sequences fill a launch; behind them only empty ones, and then one more that is not."""
    for more in ([0] * 5, [0] * 3 + [2]):
        lens = [1] * 1024 + more
        Paged(B, 2, 1, 64, [i % 9 for i in range(len(lens))], lens, "f16", page=16).check()


# ---- single tokens: several tiles of a pair in each warp --------------------------------------
# 152 SMs share the list of 64-row tiles: 120000 rows of one head are 12 tiles of 64 rows for each, and a warp
# takes every second or third of them.
LONG = 120_001


def long_step(B, Hq, hd, fmt, n=LONG, page=64, spread=1.0, q_type=None, seed=0):  # noqa: F811
    a = Paged(B, Hq, 1, hd, [n - 1], None, fmt, page=page, spread=spread, q_type=q_type, seed=seed)
    positive_values(a)
    return a


def close(a, got, ref=None):
    ref = a.ref() if ref is None else ref
    assert np.isfinite(got).all()
    err = np.abs(got - ref).max()
    assert err <= a.tol(), (err, a.tol())


@pytest.mark.parametrize("fmt", ["f16", "bf16", "e4m3"])
@pytest.mark.parametrize("Hq,hd", [(8, 64), (5, 128), (16, 64), (12, 128)])
def test_step_of_many_tiles(B, Hq, hd, fmt):  # noqa: F811
    """Scores that climb by 40 within each CTA's run and start again, that fall by as much, and that stay: the base of a warp's
    rows moves from tile to tile, and the ring's stages are used again. The same bits every time."""
    n = 200_001
    a = long_step(B, Hq, hd, fmt, n)
    base = a.c.rows[0].copy()
    ramp = np.arange(n) % 1300 / 1300 * 40                # (a run: 3126 tiles / 152 = 20.6 of 64 rows)
    for sign in (1, -1, 0):
        x = base.copy()
        x[0, :, 0, 0] = sign * (ramp + np.abs(x[0, :, 0, 1]))
        a.q[:, ::hd] = float(hd ** 0.5)                   # (element 0 of each head: its key element is the score)
        a.c.rows[0] = a.c._put(0, x)
        got = call(a)
        close(a, got)
        first = a.out.clone()
        for _ in range(3):
            a.out.fill_(55.0)
            a.call(a.ws)
            assert torch.equal(a.out, first)


@pytest.mark.parametrize("fmt", ["f16", "bf16", "e4m3"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (700, 70)])
@pytest.mark.parametrize("Hq,Hkv,hd", [(8, 2, 64), (10, 2, 128), (12, 1, 128)])
def test_step_of_many_pairs(B, Hq, Hkv, hd, window, sinks, fmt):  # noqa: F811
    """Hundreds of sequences of about a thousand rows: pairs follow one another in a CTA, each of several tiles a warp, and
    the stages go round many times."""
    g = np.random.default_rng(hd + Hq)
    pos = [int(p) for p in g.integers(600, 1500, 160)]
    pos[3], pos[7], pos[100] = -1, 0, 5000
    a = Paged(B, Hq, Hkv, hd, pos, None, fmt, page=16, window=window, sinks=sinks, spread=1.5)
    positive_values(a)
    close(a, call(a))


@pytest.mark.parametrize("Hq,hd,page,up", [(4, 128, 64, 0), (12, 64, 16, 6), (4, 64, 16, 12), (12, 128, 64, 12),
                                           (4, 128, 16, 100), (12, 64, 64, 100)])
def test_step_behind_absent_pages(B, Hq, hd, page, up):  # noqa: F811
    """8-bit pages: whole tiles without a page between ordinary ones, first in the run of many a warp; values up to 2^up
    times as large, scores wide enough that small weights make up part of the sum."""
    a = long_step(B, Hq, hd, "e4m3", page=page, spread=1.4, q_type="bf16")
    g = np.random.default_rng(up)
    tiles = np.flatnonzero(g.random(LONG // 64) < 0.4)
    tiles = np.union1d(tiles, [0, 1, 2, 3])
    per = max(1, 64 // page)
    drop_pages(a, 0, (tiles[:, None] * (64 // page) + np.arange(per)).ravel())
    scale_rows(a, 0, 1, np.arange(LONG), 2.0 ** up)
    close(a, call(a))
    # one row takes nearly all of the weight
    j = 64 * int(np.setdiff1d(np.arange(1000, 1100), tiles)[0]) + 5
    q = a.q[0, :hd].double().cpu().numpy()
    x = a.c.rows[0][:, j:j + 1].copy()
    x[0, 0, 0] = 40 * q / (q @ q) * hd ** 0.5
    a.q[:, :Hq * hd] = a.q[:, :hd].repeat(1, Hq)
    rest = a.c.rows[0]
    a.c.rows[0] = x
    places = a.c.places
    a.c.places = lambda i, n: (places(i, LONG)[0][j:j + 1], places(i, LONG)[1][j:j + 1])
    rest[:, j:j + 1] = a.c._put(0, x)
    a.c.places, a.c.rows[0] = places, rest
    close(a, call(a))


@pytest.mark.parametrize("Hq,hd,low,high", [(4, 128, -117, 0), (4, 64, -117, 110), (12, 128, -117, 110), (12, 64, -60, 20),
                                            (4, 128, -117, -60), (12, 64, -20, 4)])
def test_step_scales_that_grow(B, Hq, hd, low, high):  # noqa: F811
    """8-bit pages: tiles whose V scales lie far below those of the tiles behind them, and far above."""
    a = long_step(B, Hq, hd, "e4m3", spread=1.4, q_type="bf16")
    g = np.random.default_rng(abs(high))
    tile = np.arange(LONG) // 64
    small = (g.random(tile[-1] + 1) < 0.5)[tile]
    small[:64 * 12] = True
    scale_rows(a, 0, 1, np.flatnonzero(small), 2.0 ** low)
    scale_rows(a, 0, 1, np.flatnonzero(~small), 2.0 ** high)
    close(a, call(a))


# ---- prompts and tokens over 8-bit pages: the ends of what fp32 holds --------------------------
@pytest.mark.parametrize("up", [-100, 0, 100])
def test_prompt_behind_absent_pages(B, up):  # noqa: F811
    a = Paged(B, 4, 1, 64, [2500], [70], "e4m3", page=32, q_type="bf16", spread=1.4)
    positive_values(a)
    drop_pages(a, 0, list(range(12)) + [20, 21, 22, 23, 30, 50, 51, 52, 53])
    scale_rows(a, 0, 1, np.arange(2570), 2.0 ** up)
    close(a, call(a))


@pytest.mark.parametrize("kind", ["step", "prompt"])
@pytest.mark.parametrize("window", [0, 50])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("q_type", ["bf16", "f16"])
def test_scores_that_vanish(B, kind, window, hd, q_type):  # noqa: F811
    """Queries of zeros and small ones over tiny K scales: all scores are 0 to fp32, hidden rows stay hidden, and the result
    is the mean of the visible values."""
    for ek in (-20, -60, -116):
        a = Paged(B, 4, 1, hd, [140, 300], None if kind == "step" else [40, 200], "e4m3", page=16, window=window,
                  sinks=3 if window else 0, q_type=q_type)
        positive_values(a)
        for s in range(2):
            scale_rows(a, s, 0, np.arange(a.c.rows[s].shape[1]), 2.0 ** ek)
        a.q[::2] = 0
        a.q[1::2] *= 2.0 ** (-90 if q_type == "bf16" else -6)
        close(a, call(a))


@pytest.mark.parametrize("kind", ["step", "prompt"])
def test_scores_of_zero_times_what_fp32_does_not_hold(B, kind):  # noqa: F811
    """A query and K scales whose product passes fp32's range, the keys' codes zeros where the query is not: scores of 0."""
    a = Paged(B, 4, 1, 64, [140], None if kind == "step" else [40], "e4m3", page=16, q_type="bf16")
    positive_values(a)
    x = a.c.rows[0].copy()
    x[0, :, 0, 0] = 0
    a.c.rows[0] = a.c._put(0, x)
    scale_rows(a, 0, 0, np.arange(x.shape[1]), 2.0 ** 60)
    a.q[:] = 0
    a.q[:, ::64] = 2.0 ** 125
    close(a, call(a))


@pytest.mark.parametrize("kind", ["step", "prompt"])
@pytest.mark.parametrize("fmt", ["f16", "bf16", "e4m3"])
def test_the_largest_sm_scale(B, kind, fmt):  # noqa: F811
    """Scores of 0 at a scale that times log2 e passes fp32's range."""
    a = Paged(B, 4, 1, 64, [140], None if kind == "step" else [40], fmt, page=16)
    positive_values(a)
    a.q[:] = 0
    a.scale = 3.4e38
    close(a, call(a))


@pytest.mark.parametrize("kind", ["step", "prompt"])
@pytest.mark.parametrize("exp", [-118, -124, -130])
def test_subnormal_scales(B, kind, exp):  # noqa: F811
    """V scales below fp32's smallest normal number (2^-126) count as what they are: ordinary ones (about 2^-7) times 2^exp,
    of which fp32 keeps all bits."""
    a = Paged(B, 4, 1, 64, [400], None if kind == "step" else [40], "e4m3", page=16, q_type="bf16")
    positive_values(a)
    n = a.c.rows[0].shape[1]
    scale_rows(a, 0, 1, np.arange(n), 2.0 ** exp * np.where(np.arange(n) % 3 == 0, 1.375, 1.0))
    got, ref = call(a), a.ref()
    # besides: half a step of bf16's subnormals (2^-134); and the two joins hold means times 2^-14 l in fp32 (l: 1 .. 2), each
    # rounded by 2^-150, and divide by the sum of all these l: 2^-136 at most
    assert (np.abs(got - ref) <= a.tol() + 2.0 ** -134 + 2.0 ** -135).all()
    assert got.max() > 0


@pytest.mark.parametrize("kind", ["step", "prompt"])
@pytest.mark.parametrize("hd", [64, 128])
def test_values_near_the_largest_number(B, kind, hd):  # noqa: F811
    """V scales that bring the values to fp32's last binade: many rows of even weight, joined from many parts,
    are a mean within their range."""
    n = 60_000
    a = Paged(B, 4, 1, hd, [n], None if kind == "step" else [9], "e4m3", page=64, q_type="bf16", spread=0.5)
    positive_values(a)
    scale_rows(a, 0, 1, np.arange(a.c.rows[0].shape[1]), 2.0 ** 126)
    assert 2.0 ** 127 < a.c.rows[0][1].max() < 2.0 ** 128
    close(a, call(a))


# ---- rotations --------------------------------------------------------------------------------
def test_frequencies_of_any_size(B):  # noqa: F811
    """From a turn in 2^60 positions to 2^40 radians a position, both ways, at positions out to both ends of 32 bits."""
    g = np.random.default_rng(0)
    w = np.concatenate([2.0 ** g.uniform(-60, 40, 30) * g.choice([-1.0, 1.0], 30), [2.0 ** 40, -2.0 ** 40]])
    pos = np.array([[0, 1, -1, 2 ** 31 - 1, -2 ** 31, 77777, 2 ** 24 + 1]], np.int32)
    rows, H, hd = pos.shape[1], 2, 64
    x = torch.from_numpy(g.standard_normal((rows, H * hd))).float()
    d, p = x.cuda(), torch.from_numpy(pos).cuda()
    y = torch.empty_like(d)
    B.op_rope_async(d.data_ptr(), B.S1_F32, H * hd, rows, H, hd, B.Rope(w), p.data_ptr(), rows, y.data_ptr(), B.S1_F32, H * hd,
                    stream())
    xd = x.double().numpy().reshape(rows, H, hd)
    ref, got = rotate_ref(xd, pos, w, [0] * 32), y.double().cpu().numpy().reshape(rows, H, hd)
    tol, u, tiny = rotation_tol(xd, 32, "f32")
    assert (np.abs(got - ref) <= tol + u * np.abs(ref) + tiny).all(), np.abs(got - ref).max()
