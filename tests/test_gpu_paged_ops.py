"""The stream-ordered operators around a paged K/V cache (rotary positions, rotated append, single tokens
and prompts over pages) against their definitions in 64 bits on the CPU, on the same rounded inputs."""
import math

import numpy as np
import pytest

from test_gpu_shared_ops import E4M3, canonical, quant_ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from prefill_only_decision_gb300 import binding
    binding.lib()
    return binding


TD = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}       # half a rounding step, relative
TINY = {"f32": 2.0 ** -126, "f16": 2.0 ** -25, "bf16": 2.0 ** -126}   # (half a subnormal step, f16)


def code(B, name):
    return {"f32": B.S1_F32, "f16": B.S1_F16, "bf16": B.S1_BF16}[name]


def fmt_code(B, name):
    return {"f16": B.S1_KV_F16, "bf16": B.S1_KV_BF16, "e4m3": B.S1_KV_E4M3}[name]


def stream():
    return torch.cuda.current_stream().cuda_stream


# ---- rotary positions ------------------------------------------------------------------------
def freqs(pairs, theta=1.0e6):
    return theta ** (-np.arange(pairs) / pairs)


def rotate_ref(x, pos, w, axis):
    """x [rows, heads, hd] and pos [axes, rows] in 64 bits. Angles are reduced in integers: w as a
    fraction times the position, modulo 2 pi."""
    n = len(w)
    ang = np.empty((x.shape[0], n))
    for i in range(n):
        num, den = float(w[i]).as_integer_ratio()
        for r in range(x.shape[0]):
            p = int(pos[axis[i]][r])
            ang[r, i] = reduce_far(p * num, den)
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
    y = x.copy()
    a, b = x[..., :n], x[..., n:2 * n]
    y[..., :n], y[..., n:2 * n] = a * c - b * s, b * c + a * s
    return y


TWO_PI = 6283185307179586476925286766559005768394338798750211641949889    # 2 pi * 10^60


def reduce_far(num, den):
    """num / den radians modulo 2 pi, in integers of 60 decimals."""
    t = num * 10 ** 60 // den
    return (t % TWO_PI) / 10 ** 60


def rotation_tol(x, n, out):
    """Sine and cosine within 2^-22 (two steps of fp32, and the angle's rounding), two products and a sum of
    half a step each: 2^-21 of |a| + |b|; then one rounding to the output's type."""
    tol = np.zeros_like(x)
    m = np.abs(x[..., :n]) + np.abs(x[..., n:2 * n])
    tol[..., :n], tol[..., n:2 * n] = m, m
    return 2.0 ** -21 * tol, U[out], TINY[out]


@pytest.mark.parametrize("src,out", [("f16", "f16"), ("bf16", "bf16"), ("f32", "f32"), ("f32", "f16"), ("f32", "bf16")])
@pytest.mark.parametrize("rows,H,hd,pairs,axes,mix,pad", [
    (1, 1, 64, 8, 1, False, 0), (3, 5, 128, 64, 3, False, 8), (37, 20, 128, 64, 3, True, 16), (130, 3, 64, 32, 4, True, 1),
    (259, 2, 128, 24, 2, False, 0), (5, 300, 64, 16, 1, False, 3)])
def test_rope(B, rows, H, hd, pairs, axes, mix, pad, src, out):
    """Axes in runs and in turns, part of a head, odd strides, rows on and off 16-byte boundaries; the columns
    beside the heads stay."""
    g = np.random.default_rng(rows + H)
    x = torch.from_numpy(g.standard_normal((rows, H * hd + pad)) * np.exp(g.standard_normal((rows, 1)))).to(TD[src])
    pos = g.integers(-3000, 1_000_000, (axes, rows + 2)).astype(np.int32)
    axis = [i % axes if mix else i * axes // pairs for i in range(pairs)]
    w = freqs(pairs)
    d, p = x.cuda(), torch.from_numpy(pos).cuda()
    y = torch.full((rows, H * hd + pad), 7.0, dtype=TD[out], device="cuda")
    B.op_rope_async(d.data_ptr(), code(B, src), d.stride(0), rows, H, hd, B.Rope(w, axis, axes), p.data_ptr(),
                    p.stride(0), y.data_ptr(), code(B, out), y.stride(0), stream())
    xd = x[:, :H * hd].double().numpy().reshape(rows, H, hd)
    ref = rotate_ref(xd, pos, w, axis)
    got = y[:, :H * hd].double().cpu().numpy().reshape(rows, H, hd)
    tol, u, tiny = rotation_tol(xd, pairs, out)
    assert (np.abs(got - ref) <= tol * (1 + u) + u * np.abs(ref) + tiny).all()
    assert (y[:, H * hd:] == 7).all()
    if src == out:       # in place: the same bits
        B.op_rope_async(d.data_ptr(), code(B, src), d.stride(0), rows, H, hd, B.Rope(w, axis, axes), p.data_ptr(),
                        p.stride(0), d.data_ptr(), code(B, out), d.stride(0), stream())
        assert torch.equal(d[:, :H * hd], y[:, :H * hd]) and torch.equal(d[:, H * hd:].cpu(), x[:, H * hd:])


def test_rope_far_positions(B):
    """Positions out to both ends of 32 bits keep fp32's accuracy, and negated frequencies turn back."""
    pos = np.array([[0, 1, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 30 + 1, 123456789, -987654321, 2 ** 24 + 1]], np.int32)
    rows, H, hd, pairs = pos.shape[1], 2, 128, 64
    x = torch.from_numpy(np.random.default_rng(1).standard_normal((rows, H * hd))).float()
    w = freqs(pairs)
    d, p = x.cuda(), torch.from_numpy(pos).cuda()
    y = torch.empty_like(d)
    B.op_rope_async(d.data_ptr(), B.S1_F32, H * hd, rows, H, hd, B.Rope(w), p.data_ptr(), rows, y.data_ptr(), B.S1_F32,
                    H * hd, stream())
    xd = x.double().numpy().reshape(rows, H, hd)
    ref = rotate_ref(xd, pos, w, [0] * pairs)
    got = y.double().cpu().numpy().reshape(rows, H, hd)
    tol, u, tiny = rotation_tol(xd, pairs, "f32")
    assert (np.abs(got - ref) <= tol + u * np.abs(ref) + tiny).all(), np.abs(got - ref).max()
    B.op_rope_async(y.data_ptr(), B.S1_F32, H * hd, rows, H, hd, B.Rope(-w), p.data_ptr(), rows, y.data_ptr(), B.S1_F32,
                    H * hd, stream())
    back = y.double().cpu().numpy().reshape(rows, H, hd)
    assert (np.abs(back - xd) <= 4 * tol).all()        # two rotations, the second of values up to |a| + |b|


# ---- a paged cache on both sides -------------------------------------------------------------
def quantise(x):
    """quant_ref's codes and scales without its loop over vectors (finite values)."""
    a = np.abs(x).max(-1)
    m, e = np.frexp(a)                                     # a = m 2^e, 1/2 <= m < 1; 448 = 0.875 * 2^9
    scale = np.where(a > 0, np.exp2(np.maximum(np.where(m <= 0.875, e - 9, e - 8), -126).astype(float)), 1.0)
    y = x / scale[..., None]
    grid = E4M3[:127]
    mid = (grid[1:] + grid[:-1]) / 2
    mag = np.minimum(np.abs(y), 448.0)
    lo, hi = np.searchsorted(mid, mag, side="left"), np.searchsorted(mid, mag, side="right")
    return np.where((lo != hi) & (lo % 2 == 1), hi, lo) + 128 * np.signbit(y), scale


class Cache:
    """A pool of pages in random order. Rows that no sequence owns, the rest of each last page and spare
    pages hold NaN; table entries behind a sequence's pages hold a page id that is far out of range."""

    def __init__(self, B, ends, Hkv, hd, fmt="f16", page=16, spread=1.0, seed=0, fill=True, cols_more=2, lead_pages=0):
        self.__dict__.update(B=B, ends=list(ends), Hkv=Hkv, hd=hd, fmt=fmt, page=page)
        g = np.random.default_rng(seed + sum(ends) + 7 * Hkv + page)
        need = [(n + page - 1) // page for n in ends]
        self.n_pages = lead_pages + sum(need) + 3
        ids = lead_pages + g.permutation(self.n_pages - lead_pages)
        self.cols = max(need + [0]) + cols_more
        self.table = np.full((len(ends), self.cols + 1), 2 ** 31 - 7, np.int32)
        at = 0
        for i, n in enumerate(need):
            self.table[i, :n] = ids[at:at + n]
            at += n
        self.d_table = torch.from_numpy(self.table).cuda()
        shape = (2, self.n_pages, Hkv, page, hd)
        if fmt == "e4m3":
            self.data = torch.full(shape, 0x7f, dtype=torch.uint8, device="cuda")
            self.scales = torch.full(shape[:-1], float("nan"), device="cuda")
        else:
            self.data = torch.full(shape, float("nan"), dtype=TD[fmt], device="cuda")
            self.scales = None
        self.rows = []                                     # per sequence the 64-bit [2, n, Hkv, hd]
        for i, n in enumerate(ends):
            x = g.standard_normal((2, n, Hkv, hd)) * spread
            self.rows.append(self._put(i, x) if fill else np.zeros((2, n, Hkv, hd)))
        self.pages = B.KvPages(self.data.data_ptr(), 0 if self.scales is None else self.scales.data_ptr(),
                               fmt_code(B, fmt), self.n_pages, page, Hkv, hd, self.d_table.data_ptr(), len(self.ends),
                               self.cols, self.cols + 1)

    def places(self, i, n):
        j = np.arange(n)
        return self.table[i, j // self.page], j % self.page

    def _put(self, i, x):
        n = x.shape[1]
        if n == 0:
            return x
        pid, off = (torch.from_numpy(t.astype(np.int64)).cuda() for t in self.places(i, n))
        for plane in range(2):
            if self.fmt == "e4m3":
                c, s = quantise(x[plane])
                self.data[plane][pid, :, off] = torch.from_numpy(c.astype(np.uint8)).cuda()
                self.scales[plane][pid, :, off] = torch.from_numpy(s).float().cuda()
                x[plane] = E4M3[c] * s[..., None]
            else:
                t = torch.from_numpy(x[plane]).to(TD[self.fmt])
                self.data[plane][pid, :, off] = t.cuda()
                x[plane] = t.double().numpy()
        return x

    def set_row(self, i, j, plane, h, e, value):
        """One element of a cached row (e None: all of a head's)."""
        pid, off = int(self.table[i, j // self.page]), j % self.page
        at = slice(None) if e is None else e
        if self.fmt == "e4m3":
            assert math.isnan(value)
            self.data[plane, pid, h, off, at] = 0x7f
        else:
            self.data[plane, pid, h, off, at] = value

    def get(self, i, n):
        pid, off = (torch.from_numpy(t.astype(np.int64)).cuda() for t in self.places(i, n))
        if self.fmt != "e4m3":
            return np.stack([self.data[p][pid, :, off].double().cpu().numpy() for p in range(2)])
        return np.stack([E4M3[self.data[p][pid, :, off].cpu().numpy()] *
                         self.scales[p][pid, :, off].double().cpu().numpy()[..., None] for p in range(2)])


def visible(p, cap, window, sinks):
    j = np.arange(min(p + 1, cap) if p >= 0 else 0)
    return j[(p - j < window) | (j < sinks)] if window else j


def attend(q, kv, p, window, sinks, scale):
    """q [Hq, hd] of one row at position p over kv [2, n, Hkv, hd]."""
    Hq, Hkv = q.shape[0], kv.shape[2]
    j = visible(p, kv.shape[1], window, sinks)
    out = np.zeros(q.shape)
    if len(j) == 0:
        return out
    for h in range(Hq):
        k, v = kv[0, j, h * Hkv // Hq], kv[1, j, h * Hkv // Hq]
        z = k @ q[h] * scale
        m = z.max()
        if m == -np.inf:
            continue
        w = np.exp(z - m)
        out[h] = w @ v / w.sum()
    return out


class Paged:
    """A batch over a cache: prompts (lens rows each, starting at pos0) or single tokens (lens None)."""

    def __init__(self, B, Hq, Hkv, hd, pos0, lens=None, fmt="f16", page=16, window=0, sinks=0, gap=0, lead=0, tail=0,
                 q_type=None, seed=0, spread=1.0, **kw):
        self.__dict__.update(B=B, Hq=Hq, Hkv=Hkv, hd=hd, window=window, sinks=sinks, step=lens is None)
        self.lens = [1] * len(pos0) if lens is None else list(lens)
        self.pos0 = list(pos0)
        self.row0, at = [], lead
        for n in self.lens:
            self.row0.append(at)
            at += n + gap
        self.R = max(1, at + tail)
        self.c = Cache(B, [max(0, p + n) for p, n in zip(self.pos0, self.lens)], Hkv, hd, fmt, page, seed=seed,
                       spread=spread, **kw)
        self.q_type = q_type or ("bf16" if fmt == "bf16" else "f16")
        g = np.random.default_rng(seed + 5 + self.R)
        self.q = torch.from_numpy(g.standard_normal((self.R, Hq * hd + 8)) * spread).to(TD[self.q_type]).cuda()
        self.pos = torch.tensor(self.pos0, dtype=torch.int32, device="cuda")
        self.out = torch.full((self.R, Hq, hd), 55.0, dtype=TD[self.q_type], device="cuda")
        self.scale = hd ** -0.5

    def workspace(self):
        if self.step:
            n = self.B.op_attention_paged_step_workspace(len(self.pos0), self.Hq, self.Hkv, self.hd)
        else:
            n = self.B.op_attention_paged_workspace(self.lens, self.pos0, self.Hq, self.Hkv, self.hd, self.window,
                                                    self.sinks)
        return torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")

    def call(self, ws=None, st=None):
        self.ws = self.workspace() if ws is None else ws
        st = stream() if st is None else st
        q_type = code(self.B, self.q_type)
        if self.step:
            self.B.op_attention_paged_step_async(self.q.data_ptr(), q_type, self.q.stride(0), len(self.pos0), self.Hq,
                                                 self.c.pages, self.pos.data_ptr(), self.window, self.sinks, self.scale,
                                                 self.out.data_ptr(), self.ws.data_ptr(), self.ws.numel(), st)
        else:
            self.B.op_attention_paged_async(self.q.data_ptr(), q_type, self.q.stride(0), self.row0, self.lens, self.pos0,
                                            self.Hq, self.c.pages, self.window, self.sinks, self.scale,
                                            self.out.data_ptr(), self.ws.data_ptr(), self.ws.numel(), st)

    def ref(self, rows=None):
        out = np.full((self.R, self.Hq, self.hd), 55.0)
        q = self.q[:, :self.Hq * self.hd].double().cpu().numpy().reshape(self.R, self.Hq, self.hd)
        for s, (r0, n, p0) in enumerate(zip(self.row0, self.lens, self.pos0)):
            for i in range(n):
                if rows is None or r0 + i in rows:
                    out[r0 + i] = attend(q[r0 + i], self.c.rows[s], p0 + i, self.window, self.sinks, self.scale)
        return out

    def tol(self):
        """The weights are rounded to the product's type (f16 beside e4m3 pages), so at most half a step of it
        of max |v| in a weighted mean, the result once to its own; fp32 scores of at most a few hundred terms and
        exp move a weight by less than 2^-13 at these score sizes."""
        v = max([np.abs(np.nan_to_num(r[1], nan=0, posinf=0, neginf=0)).max() for r in self.c.rows if r.size] + [0.0])
        w = U["bf16"] if self.c.fmt == "bf16" else U["f16"]
        return (w + U[self.q_type] + 2.0 ** -12) * v

    def check(self):
        self.call()
        self.B.op_sync(stream())
        got, ref = self.out.double().cpu().numpy(), self.ref()
        err = np.abs(got - ref).max()
        assert err <= self.tol(), (err, self.tol())          # (rows of no sequence: 55 on both sides)


# ---- rows appended to pages ------------------------------------------------------------------
def append_case(B, lens, first, Hq, Hkv, hd, src, fmt, page, axes, pad, seq=True, rope=True, q_type=None, pos=True):
    ends = [a + n for a, n in zip(first, lens)]
    c = Cache(B, ends, Hkv, hd, fmt, page, fill=False)
    rows = sum(lens)
    g = np.random.default_rng(rows + Hkv)
    W = (Hq + 2 * Hkv) * hd
    x = torch.from_numpy(g.standard_normal((rows, W + pad)) * np.exp(2 * g.standard_normal((rows, 1)))).to(TD[src])
    d = x.cuda()
    owner = np.repeat(np.arange(len(lens)), lens).astype(np.int32)
    at = np.concatenate([np.arange(a, a + n) for a, n in zip(first, lens)]).astype(np.int32)
    p = g.integers(0, 200_000, (axes, rows)).astype(np.int32) if pos else np.stack([at] * axes)
    w = freqs(hd // 2)
    axis = [i % axes for i in range(hd // 2)]
    q_type = q_type or ("bf16" if fmt == "bf16" else "f16")
    q_out = torch.full((rows, Hq * hd), 9.0, dtype=TD[q_type], device="cuda")
    t = [torch.from_numpy(a).cuda() for a in (owner, at, p)]
    es = d.element_size()
    B.op_kv_append_async(d.data_ptr() if Hq else 0, d.data_ptr() + Hq * hd * es, d.data_ptr() + (Hq + Hkv) * hd * es,
                         code(B, src), d.stride(0), d.stride(0), d.stride(0), rows, Hq,
                         B.Rope(w, axis, axes) if rope else None, t[2].data_ptr() if pos else 0, rows,
                         t[0].data_ptr() if seq else 0, t[1].data_ptr(), c.pages, q_out.data_ptr() if Hq else 0,
                         code(B, q_type), stream())
    xd = x[:, :W].double().numpy().reshape(rows, -1, hd)
    turned = rotate_ref(xd[:, :Hq + Hkv], p, w, axis) if rope else xd[:, :Hq + Hkv]
    tol, u, tiny = rotation_tol(xd[:, :Hq + Hkv], hd // 2, q_type)
    if not rope:
        tol = 0 * tol
    got = q_out.double().cpu().numpy().reshape(rows, Hq, hd)
    assert (np.abs(got - turned[:, :Hq]) <= tol[:, :Hq] * (1 + u) + u * np.abs(turned[:, :Hq]) + tiny).all()
    k_ref, k_tol, v_ref = turned[:, Hq:], tol[:, Hq:], xd[:, Hq + Hkv:]
    written = np.zeros((c.n_pages, page), bool)
    r = 0
    for i, (a, n) in enumerate(zip(first, lens)):
        pid, off = (z[a:] for z in c.places(i, a + n))
        written[pid, off] = True
        P = torch.from_numpy(pid.astype(np.int64)).cuda()
        O = torch.from_numpy(off.astype(np.int64)).cuda()
        kr, kt, vr = k_ref[r:r + n], k_tol[r:r + n], v_ref[r:r + n]
        if fmt == "e4m3":
            kc, vc = (c.data[j][P, :, O].cpu().numpy() for j in range(2))
            ks, vs = (c.scales[j][P, :, O].double().cpu().numpy() for j in range(2))
            rc, rs = quant_ref(vr)
            assert np.array_equal(canonical(vc), canonical(rc)) and np.array_equal(vs, rs)
            top = np.abs(kr).max(-1)                       # the scale of a maximum within its error
            lo = quant_ref(np.maximum(top - kt.max(-1), 0)[..., None])[1]
            hi = quant_ref((top + kt.max(-1))[..., None])[1]
            assert ((ks == lo) | (ks == hi)).all()
            # half a step: 2^-4 of the value, or 2^-10 of the scale below the normal codes
            val = E4M3[kc] * ks[..., None]
            assert (np.abs(val - kr) <= np.maximum(2.0 ** -4 * (np.abs(kr) + kt), 2.0 ** -10 * ks[..., None]) + kt).all()
        else:
            u = U[fmt]
            kg, vg = (c.data[j][P, :, O].double().cpu().numpy() for j in range(2))
            assert (np.abs(kg - kr) <= kt * (1 + u) + u * np.abs(kr) + TINY[fmt]).all()
            assert np.array_equal(vg, torch.from_numpy(vr).to(TD[fmt]).double().numpy())
        r += n
    left = torch.from_numpy(~written).cuda()
    for j in range(2):                                      # every other row of the pool is as it was
        rest = c.data[j].transpose(1, 2)[left]
        assert (rest == 0x7f).all() if fmt == "e4m3" else torch.isnan(rest).all()
        if fmt == "e4m3":
            assert torch.isnan(c.scales[j].transpose(1, 2)[left]).all()


@pytest.mark.parametrize("src", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("fmt", ["f16", "bf16", "e4m3"])
@pytest.mark.parametrize("lens,first,Hq,Hkv,hd,page,axes,pad", [
    ([1], [0], 1, 1, 64, 16, 1, 0), ([1] * 7, [0, 15, 16, 17, 300, 31, 63], 16, 4, 128, 16, 1, 8),
    ([3, 40, 1], [0, 100, 9], 6, 2, 64, 32, 3, 1), ([130, 65], [5, 127], 10, 2, 128, 64, 3, 24),
    ([257], [128], 4, 4, 64, 128, 2, 0)])
def test_append(B, lens, first, Hq, Hkv, hd, page, axes, pad, fmt, src):
    append_case(B, lens, first, Hq, Hkv, hd, src, fmt, page, axes, pad)


@pytest.mark.parametrize("kw", [dict(seq=False), dict(pos=False), dict(rope=False), dict(seq=False, pos=False, fmt="e4m3",
                                                                                          q_type="bf16")])
def test_append_defaults(B, kw):
    """No sequence numbers (row i is sequence i's), no positions (the rows' own), no rotation."""
    fmt = kw.pop("fmt", "f16")
    append_case(B, [1] * 5, [0, 3, 16, 40, 33], 8, 2, 128, "f16", fmt, 16, 1, 0, **kw)


def test_append_without_queries(B):
    append_case(B, [9, 30], [1, 0], 0, 3, 64, "f32", "bf16", 16, 2, 4)


def test_append_special_values(B):
    """NaN and infinities travel as the formats hold them; e4m3 takes its scale from the finite ones."""
    rows, Hkv, hd = 4, 1, 64
    v = torch.ones(rows, hd)
    v[0, 3], v[1, 5], v[2, :], v[3, :] = float("nan"), float("inf"), -float("inf"), 0.0
    x = v.cuda()
    for fmt in ("f16", "bf16", "e4m3"):
        c = Cache(B, [rows], Hkv, hd, fmt, 16, fill=False)
        at = torch.arange(rows, dtype=torch.int32, device="cuda")
        own = torch.zeros(rows, dtype=torch.int32, device="cuda")
        B.op_kv_append_async(0, x.data_ptr(), x.data_ptr(), B.S1_F32, 0, hd, hd, rows, 0, None, 0, 0, own.data_ptr(),
                             at.data_ptr(), c.pages, 0, B.S1_F16, stream())
        pid = int(c.table[0, 0])
        for plane in range(2):
            if fmt == "e4m3":
                rc, rs = quant_ref(v.double().numpy())
                assert np.array_equal(canonical(c.data[plane, pid, 0, :rows].cpu().numpy()), canonical(rc))
                assert np.array_equal(c.scales[plane, pid, 0, :rows].cpu().numpy(), rs)
            else:
                got = c.data[plane, pid, 0, :rows].float().cpu()
                assert torch.equal(torch.nan_to_num(got, nan=9.0), torch.nan_to_num(v, nan=9.0))


def test_append_padding_and_places_that_do_not_exist(B):
    """Padding rows write nothing; a sequence, a row or a page outside what there is drops k and v but not q."""
    Hq, Hkv, hd, page = 4, 2, 64, 16
    c = Cache(B, [20, 20], Hkv, hd, "f16", page, fill=False, cols_more=1)
    c.d_table[1, 0], c.d_table[1, 1] = -1, c.n_pages                # bad pages within sequence 1
    before = c.data.clone()
    cases = [(0, -1), (2, 0), (-1, 0), (0, c.cols * page), (0, 2 ** 31 - 1), (1, 0), (1, 16), (0, 40), (0, -2 ** 31)]
    rows = len(cases)
    x = torch.randn(rows, (Hq + 2 * Hkv) * hd, device="cuda").half()
    own, at = (torch.tensor(t, dtype=torch.int32, device="cuda") for t in zip(*cases))
    q_out = torch.full((rows, Hq * hd), 9.0, dtype=torch.float16, device="cuda")
    B.op_kv_append_async(x.data_ptr(), x.data_ptr() + Hq * hd * 2, x.data_ptr() + (Hq + Hkv) * hd * 2, B.S1_F16,
                         x.stride(0), x.stride(0), x.stride(0), rows, Hq, None, 0, 0, own.data_ptr(), at.data_ptr(),
                         c.pages, q_out.data_ptr(), B.S1_F16, stream())
    assert torch.equal(torch.nan_to_num(c.data, nan=1e4), torch.nan_to_num(before, nan=1e4))
    for i, (_, a) in enumerate(cases):
        assert (q_out[i] == 9).all() if a < 0 else torch.equal(q_out[i], x[i, :Hq * hd])


# ---- attention over pages --------------------------------------------------------------------
WINDOWS = [(0, 0), (1, 0), (5, 2), (64, 4), (200, 130), (1000000, 7)]
STEPS = [  # Hq, Hkv, hd, page, positions
    (1, 1, 64, 16, [0]), (16, 4, 128, 16, [1023, 999, 1040]), (40, 8, 128, 64, [0, 15, 16, 63, 64, 127, 700]),
    (4, 4, 128, 32, [31, 32, 33, 500]), (16, 1, 64, 128, [127, 128, 129]), (17, 1, 128, 16, [300]),
    (128, 1, 64, 64, [77, 260]), (6, 2, 64, 16, [-1, 5, -1, 2000, -7]), (12, 3, 128, 128, [4000])]


@pytest.mark.parametrize("fmt", ["f16", "bf16", "e4m3"])
@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("Hq,Hkv,hd,page,pos", STEPS)
def test_step(B, Hq, Hkv, hd, page, pos, window, sinks, fmt):
    Paged(B, Hq, Hkv, hd, pos, None, fmt, page, window, sinks).check()


PROMPTS = [  # Hq, Hkv, hd, page, lens, pos0
    (1, 1, 64, 16, [1], [0]), (16, 4, 128, 16, [300], [0]), (8, 2, 64, 64, [1, 0, 129, 33], [0, 9, 200, 511]),
    (40, 8, 128, 32, [30, 64], [127, 1]), (4, 4, 128, 128, [257], [128]), (17, 1, 64, 16, [9, 20], [700, 0]),
    (128, 1, 128, 64, [3], [90]), (6, 2, 128, 16, [0, 140, 0], [5, 1000, 0])]


@pytest.mark.parametrize("fmt", ["f16", "bf16", "e4m3"])
@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("Hq,Hkv,hd,page,lens,pos0", PROMPTS)
def test_prompt(B, Hq, Hkv, hd, page, lens, pos0, window, sinks, fmt):
    Paged(B, Hq, Hkv, hd, pos0, lens, fmt, page, window, sinks, gap=3, lead=2, tail=1).check()


@pytest.mark.parametrize("kind", ["step", "prompt"])
def test_bf16_queries_over_8_bit_pages(B, kind):
    """Queries far outside f16's range keep their bits: 2^40 with scores brought back by sm_scale."""
    for mag in (1.0, 2.0 ** 40, 2.0 ** -40):
        a = Paged(B, 8, 2, 128, [300, 40, 7], None if kind == "step" else [5, 70, 130], "e4m3", q_type="bf16")
        a.q *= mag
        a.scale /= mag
        a.check()


@pytest.mark.parametrize("kind", ["step", "prompt"])
def test_8_bit_scales_out_of_the_ordinary(B, kind):
    """Rows whose scales lie far from one another (2^-60 to 2^20), and scales that are no powers of two."""
    a = Paged(B, 8, 2, 64, [300], None if kind == "step" else [70], "e4m3", page=16)
    pid, off = (torch.from_numpy(t.astype(np.int64)).cuda() for t in a.c.places(0, len(a.c.rows[0][0])))
    n = len(off)
    g = np.random.default_rng(3)
    for plane, e in ((0, g.integers(-60, 3, (n, 2))), (1, g.integers(-60, 20, (n, 2)))):
        f = 2.0 ** e * np.where(np.arange(n) % 3 == 0, 1.375, 1.0)[:, None]
        a.c.scales[plane][pid, :, off] *= torch.from_numpy(f).float().cuda()
        a.c.rows[0][plane] *= f[..., None]
    a.call()
    # values of up to 448 * 1.375 * 2^20 pass f16's largest number: a result past 65520 rounds to infinity, so both sides
    # are held at 65504, which moves neither closer to the other by more than that rounding
    got, ref = (np.clip(t, -65504, 65504) for t in (a.out.double().cpu().numpy(), a.ref()))
    # the weights' rounding: relative to the largest contribution, w |v|, which max |v| bounds
    assert not np.isnan(got).any() and (np.abs(got - ref) <= a.tol()).all()


@pytest.mark.parametrize("kind", ["step", "prompt"])
def test_8_bit_scales_at_the_ends_of_their_range(B, kind):
    """All K scales near fp32's smallest (the queries bring the scores back) and V scales near its smallest or largest, bf16."""
    for ek, ev in ((-116, -110), (-100, 112), (90, 0)):
        a = Paged(B, 4, 1, 64, [140], None if kind == "step" else [40], "e4m3", page=16, q_type="bf16")
        pid, off = (torch.from_numpy(t.astype(np.int64)).cuda() for t in a.c.places(0, len(a.c.rows[0][0])))
        for plane, e in ((0, ek), (1, ev)):
            a.c.scales[plane][pid, :, off] *= 2.0 ** e
            a.c.rows[0][plane] *= 2.0 ** e
        a.q *= 2.0 ** -ek
        a.check()


@pytest.mark.parametrize("kind", ["step", "prompt"])
@pytest.mark.parametrize("fmt", ["f16", "bf16", "e4m3"])
def test_hidden_rows_do_not_matter(B, kind, fmt):
    """NaN in keys and values that a window hides, or that lie ahead, reaches only the rows that see them."""
    lens = None if kind == "step" else [200, 60]
    a = Paged(B, 8, 2, 64, [400, 333], lens, fmt, page=32, window=100, sinks=3)
    clean = a.ref()
    bad = [3, 60, 250, 301] if kind == "step" else [3, 60, 250, 300, 301, 420, 507, 599]
    for j in bad:
        for plane in range(2):
            a.c.set_row(0, j, plane, 0, None, float("nan"))
    a.call()
    got = a.out.double().cpu().numpy()
    seen = np.zeros(a.R, bool)
    n0 = a.lens[0]
    for i in range(n0):
        seen[a.row0[0] + i] = bool(np.isin(visible(a.pos0[0] + i, 10 ** 6, 100, 3), bad).any())
    assert kind == "step" or (seen.any() and not seen[:n0].all())
    assert (np.abs(got - clean)[~seen] <= a.tol()).all()
    assert (np.abs(got - clean)[seen][:, 4:] <= a.tol()).all()        # the other kv head
    assert np.isnan(got[seen][:, :4]).all()


@pytest.mark.parametrize("kind", ["step", "prompt"])
@pytest.mark.parametrize("fmt", ["f16", "bf16"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_nonfinite_values(B, kind, fmt, bad):
    """An element of a value row that is not finite reaches its own column of the rows that see it."""
    a = Paged(B, 4, 2, 128, [130, 50], None if kind == "step" else [150, 9], fmt, window=90, sinks=1)
    a.c.rows[0][0] *= 0.25                                 # (no weight so small that it is zero)
    a.c._put(0, a.c.rows[0].copy())
    clean = a.ref()
    j = 101
    a.c.set_row(0, j, 1, 1, 9, bad)
    a.call()
    got = a.out.double().cpu().numpy()
    hit = np.zeros(got.shape, bool)
    for i in range(a.lens[0]):
        if j in visible(a.pos0[0] + i, 10 ** 6, 90, 1):
            hit[a.row0[0] + i, 2:, 9] = True
    assert hit.any() and (np.abs(got - clean)[~hit] <= a.tol()).all()
    assert np.isnan(got[hit]).all() if math.isnan(bad) else (got[hit] == bad).all()


@pytest.mark.parametrize("kind", ["step", "prompt"])
def test_scores_of_minus_infinity(B, kind):
    """A query all of whose scores are -inf gives zeros; -inf among others drops out."""
    a = Paged(B, 2, 1, 64, [40, 30], None if kind == "step" else [1, 1], "f16")
    a.q[:, :] = 0
    a.q[:, 0], a.q[:, 64] = 1.0, 1.0
    for j in range(41):
        a.c.set_row(0, j, 0, 0, 0, -float("inf"))
    a.c.set_row(1, 3, 0, 0, 0, -float("inf"))
    a.c.rows[1][0, 3, 0, 0] = -np.inf
    a.c.rows[0][0, :, 0, 0] = -np.inf
    a.call()
    got = a.out.double().cpu().numpy()
    assert (got[a.row0[0]] == 0).all()
    assert np.abs(got[a.row0[1]] - a.ref()[a.row0[1]]).max() <= a.tol()


@pytest.mark.parametrize("kind", ["step", "prompt"])
@pytest.mark.parametrize("fmt", ["f16", "e4m3"])
def test_bad_pages_read_as_zeros(B, kind, fmt):
    a = Paged(B, 8, 2, 64, [200], None if kind == "step" else [40], fmt, page=32)
    for col, pid in ((1, -1), (3, a.c.n_pages), (4, 2 ** 31 - 1), (5, -2 ** 31)):
        a.c.d_table[0, col] = pid
        a.c.rows[0][:, col * 32:(col + 1) * 32] = 0
    a.check()


def test_step_positions_past_the_table(B):
    """A token beyond the table's rows sees those that there are."""
    a = Paged(B, 8, 2, 64, [63, 31], None, "f16", page=32, window=40, sinks=2, cols_more=0)
    for p in (64, 70, 102, 103, 104, 5000, 2 ** 31 - 1):
        a.pos[0] = p
        a.pos0[0] = p
        a.check()


@pytest.mark.parametrize("kind", ["step", "prompt"])
@pytest.mark.parametrize("fmt", ["f16", "bf16", "e4m3"])
def test_growing_maxima_and_sinks(B, kind, fmt):
    """Scores that grow along the keys, and a first row that takes nearly all the weight: the rest keeps its bits."""
    a = Paged(B, 4, 1, 64, [900], None if kind == "step" else [30], fmt, window=0)
    base = a.c.rows[0].copy()
    for sign, sink in ((1, False), (-1, False), (0, True)):
        x = base.copy()
        q = torch.zeros_like(a.q)
        q[:, ::64] = 1.0
        n = x.shape[1]
        x[0, :, 0, 0] = sign * np.arange(n) * 0.25
        if sink:                                            # e^14 above the others, its value zero
            x[0, 0, 0, 0] = 112.0
            x[1, 0] = 0.0
        a.q = q
        a.c.rows[0] = a.c._put(0, x)
        a.call()
        got, ref = a.out.double().cpu().numpy(), a.ref()
        tol = a.tol()
        if sink:     # relative to the outputs, which are about 900 e^-14 of the values
            w = U["bf16"] if fmt == "bf16" else U["f16"]
            share = 930 * math.exp(-14.0)
            tol = (w + U[a.q_type] + 2.0 ** -12) * share * np.abs(x[1]).max() + (2.0 ** -24 if a.q_type == "f16" else 0)
        assert np.abs(got - ref).max() <= tol


@pytest.mark.parametrize("n", [300, 1500])
def test_many_sequences(B, n):
    g = np.random.default_rng(n)
    pos = [int(p) for p in g.integers(-3, 40, n)]
    Paged(B, 2, 1, 64, pos, None, "f16", page=16, window=9, sinks=1).check()
    Paged(B, 2, 1, 64, [max(0, p) for p in pos], [int(x) for x in g.integers(0, 4, n)], "f16", page=16).check()


def test_step_with_few_active_sequences(B):
    """Thousands of padding tokens between the ones that see something."""
    for n, active in ((3000, [7, 8, 1200, 2999]), (200, [199]), (257, [0, 256]), (40, [])):
        pos = [-1 - i % 3 for i in range(n)]
        for k, i in enumerate(active):
            pos[i] = 700 * k + 3
        Paged(B, 6, 3, 64, pos, None, "f16", page=16).check()


def sampled(a, rows):
    """check() for some rows; all others of a sequence finite."""
    a.call()
    a.B.op_sync(stream())
    got, ref = a.out.double().cpu().numpy(), a.ref(set(rows))
    assert np.abs(got[rows] - ref[rows]).max() <= a.tol() and np.isfinite(got).all()


@pytest.mark.parametrize("fmt", ["f16", "bf16", "e4m3"])
def test_prompt_of_many_items(B, fmt):
    """More items than a few per SM, of two query tiles (one long sequence), of one (many short ones), and of both lengths
    with the long ones' keys split."""
    g = np.random.default_rng(4)
    a = Paged(B, 128, 8, 64, [0], [6000], fmt, page=64, window=40, sinks=2)
    sampled(a, [0, 7, 8, 15, 16, 39, 40, 41, 127, 128] + [int(r) for r in g.integers(0, 6000, 20)] + [5999])
    lens = [int(x) for x in g.integers(1, 60, 150)]
    a = Paged(B, 32, 32, 64, [int(x) for x in g.integers(0, 300, 150)], lens, fmt, page=16, gap=1)
    rows = sorted(int(a.row0[s] + g.integers(0, lens[s])) for s in range(0, 150, 5))
    sampled(a, rows)
    Paged(B, 8, 2, 128, [20000, 0, 7, 15000], [5, 300, 2, 40], fmt, page=32, gap=2).check()


@pytest.mark.parametrize("kind", ["step", "prompt"])
def test_sequences_that_share_pages(B, kind):
    """Two sequences whose tables name the same pages see the same rows."""
    a = Paged(B, 8, 2, 64, [300, 300], None if kind == "step" else [40, 40], "f16", page=32)
    a.c.d_table[1] = a.c.d_table[0]
    a.c.rows[1] = a.c.rows[0]
    a.check()


@pytest.mark.parametrize("fmt", ["f16", "e4m3"])
def test_long_caches_split_and_repeat(B, fmt):
    """Few rows over a long cache are split over the SMs; the same bits every time."""
    for lens in (None, [5]):
        a = Paged(B, 4, 1, 128, [20001], lens, fmt, page=64)
        a.check()
        first = a.out.clone()
        for _ in range(5):
            a.out.fill_(55.0)
            a.call(a.ws)
            assert torch.equal(a.out, first)


def test_step_captured_as_positions_grow(B):
    """One captured call of append and attention follows the positions, tables and rows it finds at replay."""
    Hq, Hkv, hd, n = 8, 2, 128, 3
    a = Paged(B, Hq, Hkv, hd, [30, 500, 63], None, "f16", page=16, fill=True, cols_more=4)
    W = (Hq + 2 * Hkv) * hd
    x = torch.zeros(n, W, dtype=torch.float16, device="cuda")
    q = torch.zeros(n, Hq * hd, dtype=torch.float16, device="cuda")
    w = freqs(hd // 2)
    rope = B.Rope(w)
    ws = a.workspace()
    # the pages that the sequences grow into
    spare = [p for p in range(a.c.n_pages) if p not in a.c.table[a.c.table < a.c.n_pages]]
    a.c.table[0, 2], a.c.table[2, 4] = spare[0], spare[1]
    a.c.d_table.copy_(torch.from_numpy(a.c.table))
    side = torch.cuda.Stream()

    def calls():
        st = torch.cuda.current_stream().cuda_stream
        B.op_kv_append_async(x.data_ptr(), x.data_ptr() + Hq * hd * 2, x.data_ptr() + (Hq + Hkv) * hd * 2, B.S1_F16, W, W,
                             W, n, Hq, rope, 0, 0, 0, a.pos.data_ptr(), a.c.pages, q.data_ptr(), B.S1_F16, st)
        B.op_attention_paged_step_async(q.data_ptr(), B.S1_F16, Hq * hd, n, Hq, a.c.pages, a.pos.data_ptr(), 0, 0, a.scale,
                                        a.out.data_ptr(), ws.data_ptr(), ws.numel(), st)

    with torch.cuda.stream(side):
        calls()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    g = np.random.default_rng(0)
    for t in range(4):
        pos = [31 + t, 501 + t, -1 if t == 2 else 64 + t - (t > 2)]
        x.copy_(torch.from_numpy(g.standard_normal((n, W))).half())
        a.pos.copy_(torch.tensor(pos, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        xd = x.double().cpu().numpy().reshape(n, -1, hd)
        qr = q.double().cpu().numpy().reshape(n, Hq, hd)
        for s, p in enumerate(pos):
            if p < 0:
                assert (a.out[s] == 0).all()
                continue
            kv = a.c.get(s, p + 1)
            k = rotate_ref(xd[s:s + 1, Hq:Hq + Hkv], [[p]], w, [0] * (hd // 2))[0]
            assert np.abs(kv[0, p] - k).max() <= 2.0 ** -10 * np.abs(k).max()
            assert np.array_equal(kv[1, p], xd[s, Hq + Hkv:])
            ref = attend(qr[s], kv, p, 0, 0, a.scale)
            assert np.abs(a.out[s].double().cpu().numpy() - ref).max() <= (2 * 2.0 ** -11 + 2.0 ** -12) * np.abs(kv[1]).max()


def test_calls_at_once(B):
    """Calls on two streams, eager and as graphs, with a workspace each."""
    mk = [lambda: Paged(B, 16, 4, 128, [3000, 17, 900], None, "f16", page=16, seed=1),
          lambda: Paged(B, 16, 4, 128, [2000], [70], "f16", page=32, seed=2, window=700, sinks=4),
          lambda: Paged(B, 8, 1, 64, [5000], None, "e4m3", page=128, seed=3),
          lambda: Paged(B, 8, 1, 64, [4000], [33], "e4m3", page=64, seed=4)]
    runs = [f() for f in mk]
    refs = [r.ref() for r in runs]
    for r in runs:
        r.call()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    graphs = []
    for r, st in zip(runs, streams):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=st):
            r.call(r.ws, st.cuda_stream)
        graphs.append(gr)
    for mode in ("eager", "graph"):
        for r in runs:
            r.out.fill_(55.0)
        torch.cuda.synchronize()
        for _ in range(10):
            for r, st, gr in zip(runs, streams, graphs):
                with torch.cuda.stream(st):
                    r.call(r.ws, st.cuda_stream) if mode == "eager" else gr.replay()
        torch.cuda.synchronize()
        for r, ref in zip(runs, refs):
            assert np.abs(r.out.double().cpu().numpy() - ref).max() <= r.tol()


@pytest.mark.parametrize("fmt", ["f16", "e4m3"])
def test_offsets_past_32_bits(B, fmt):
    """Pages whose elements and bytes lie beyond 2^32 of the cache's start, in both planes."""
    Hkv, hd, page = 2, 128, 128
    lead = (1 << 32) // (Hkv * hd * page) + 1               # elements before the used pages
    a = Paged(B, 8, Hkv, hd, [300, 5], None, fmt, page=page, lead_pages=lead)
    a.check()
    b = Paged(B, 8, Hkv, hd, [200], [40], fmt, page=page, lead_pages=lead)
    b.check()
    del a, b
    append_far(B, fmt, lead, Hkv, hd, page)


def append_far(B, fmt, lead, Hkv, hd, page):
    c = Cache(B, [140], Hkv, hd, fmt, page, fill=False, lead_pages=lead)
    x = torch.randn(140, 2 * Hkv * hd, device="cuda").half()
    at = torch.arange(140, dtype=torch.int32, device="cuda")
    own = torch.zeros(140, dtype=torch.int32, device="cuda")
    B.op_kv_append_async(0, x.data_ptr(), x.data_ptr() + Hkv * hd * 2, B.S1_F16, 0, x.stride(0), x.stride(0), 140, 0, None,
                         0, 0, own.data_ptr(), at.data_ptr(), c.pages, 0, B.S1_F16, stream())
    got = c.get(0, 140)
    ref = x.double().cpu().numpy().reshape(140, 2, Hkv, hd).transpose(1, 0, 2, 3)
    tol = 2.0 ** -4 * np.abs(ref) + 2.0 ** -9 if fmt == "e4m3" else 0    # (scales of at most 2^-6 here)
    assert (np.abs(got - ref) <= tol).all()


# ---- together --------------------------------------------------------------------------------
@pytest.mark.parametrize("fmt", ["f16", "bf16", "e4m3"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (48, 4)])
def test_prompts_then_tokens(B, fmt, window, sinks):
    """Ragged multimodal prompts go through rotation and pages in two chunks, then tokens one by one; the outputs follow
    from what the cache holds, and the cache from the projections' rows."""
    Hq, Hkv, hd, page, axes = 10, 2, 128, 16, 3
    total = [100, 37, 1]                                    # rows of the prompts; then 3 tokens each
    dt = "bf16" if fmt == "bf16" else "f16"
    c = Cache(B, [n + 3 for n in total], Hkv, hd, fmt, page, fill=False)
    w, axis = freqs(hd // 2), [i % axes for i in range(hd // 2)]
    rope = B.Rope(w, axis)
    g = np.random.default_rng(0)
    W = (Hq + 2 * Hkv) * hd
    done = [0] * 3
    u = U["bf16"] if fmt == "bf16" else U["f16"]
    for chunk in ([60, 37, 0], [40, 0, 1], [1, 1, 1], [1, 1, 1], [1, 1, 1]):
        rows = sum(chunk)
        x = torch.from_numpy(g.standard_normal((rows, W))).to(TD[dt]).cuda()
        own = np.repeat(np.arange(3), chunk).astype(np.int32)
        at = np.concatenate([np.arange(d, d + n) for d, n in zip(done, chunk)]).astype(np.int32)
        pos = np.stack([at, at // 9, at % 9]).astype(np.int32)
        t = [torch.from_numpy(z).cuda() for z in (own, at, pos)]
        q = torch.empty(rows, Hq * hd, dtype=TD[dt], device="cuda")
        out = torch.empty(rows, Hq, hd, dtype=TD[dt], device="cuda")
        es = x.element_size()
        B.op_kv_append_async(x.data_ptr(), x.data_ptr() + Hq * hd * es, x.data_ptr() + (Hq + Hkv) * hd * es, code(B, dt), W, W,
                             W, rows, Hq, rope, t[2].data_ptr(), rows, t[0].data_ptr(), t[1].data_ptr(), c.pages,
                             q.data_ptr(), code(B, dt), stream())
        row0 = [int(v) for v in np.cumsum([0] + chunk[:-1])]
        if chunk == [1, 1, 1]:
            ws = torch.empty(max(16, B.op_attention_paged_step_workspace(3, Hq, Hkv, hd)), dtype=torch.uint8, device="cuda")
            B.op_attention_paged_step_async(q.data_ptr(), code(B, dt), Hq * hd, 3, Hq, c.pages, t[1].data_ptr(), window, sinks,
                                            hd ** -0.5, out.data_ptr(), ws.data_ptr(), ws.numel(), stream())
        else:
            nb = B.op_attention_paged_workspace(chunk, done, Hq, Hkv, hd, window, sinks)
            ws = torch.empty(max(16, nb), dtype=torch.uint8, device="cuda")
            B.op_attention_paged_async(q.data_ptr(), code(B, dt), Hq * hd, row0, chunk, done, Hq, c.pages, window, sinks,
                                       hd ** -0.5, out.data_ptr(), ws.data_ptr(), ws.numel(), stream())
        B.op_sync(stream())
        xd = x.double().cpu().numpy().reshape(rows, -1, hd)
        qd, od = q.double().cpu().numpy().reshape(rows, Hq, hd), out.double().cpu().numpy()
        turned = rotate_ref(xd[:, :Hq + Hkv], pos, w, axis)
        assert np.abs(qd - turned[:, :Hq]).max() <= 1.1 * U[dt] * np.abs(turned).max()
        for s in range(3):
            kv = c.get(s, done[s] + chunk[s])
            for i in range(chunk[s]):
                r = row0[s] + i
                step = 2.0 ** -4 if fmt == "e4m3" else 1.1 * U[dt]
                assert np.abs(kv[0, done[s] + i] - turned[r, Hq:]).max() <= step * np.abs(turned).max()
                ref = attend(qd[r], kv, done[s] + i, window, sinks, hd ** -0.5)
                assert np.abs(od[r] - ref).max() <= (u + U[dt] + 2.0 ** -12) * np.abs(kv[1]).max()
        done = [d + n for d, n in zip(done, chunk)]
