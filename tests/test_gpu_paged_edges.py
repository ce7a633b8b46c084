"""The paged operators where several tiles of a sequence meet in one warp: bases and units that move, stages that
are used again, pages that are not there, scales at the ends of their range. Against the definitions in 64 bits."""
import numpy as np
import pytest

from test_gpu_paged_ops import B, Paged, stream  # noqa: F401  (B: the fixture)

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
