"""The stream-ordered operators over a long shared prefix (8-bit K/V snapshot, attention of a
batch over one prefix, linear attention with a decay per head) against their definitions in 64
bits on the CPU, on the same rounded inputs."""
import math

import numpy as np
import pytest

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
U = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}       # half a rounding step, relative


def code(B, name):
    return {"f32": B.S1_F32, "f16": B.S1_F16, "bf16": B.S1_BF16}[name]


def stream():
    return torch.cuda.current_stream().cuda_stream


# ---- the 8-bit snapshot ----------------------------------------------------------------------
def e4m3_value(b):
    """The value of e4m3 bytes (sign, 4 exponent bits of bias 7, 3 mantissa bits; 0x7f is NaN)."""
    b = b.astype(np.int64)
    e, m = (b >> 3) & 15, b & 7
    x = np.where(e > 0, (8 + m) * 2.0 ** (e - 10), m * 2.0 ** -9)
    x = np.where((b & 127) == 127, np.nan, x)
    return np.where(b >> 7, -x, x)


E4M3 = e4m3_value(np.arange(256))


def quant_ref(x):
    """Codes and scales of [..., hd] float64 vectors: the nearest of the 253 finite values, ties to
    the even code, found by comparing with all midpoints."""
    fin = np.where(np.isfinite(x), np.abs(x), 0.0)
    a = fin.max(-1)
    scale = np.ones_like(a)
    for i in np.ndindex(a.shape):
        if a[i] > 0:
            E = -126
            while 448.0 * 2.0 ** E < a[i]:
                E += 1
            scale[i] = 2.0 ** E
    y = x / scale[..., None]
    grid = E4M3[:127]                              # 0 .. 448, ascending
    mid = (grid[1:] + grid[:-1]) / 2
    mag = np.minimum(np.abs(np.nan_to_num(y, nan=0.0, posinf=448, neginf=-448)), 448.0)
    lo = np.searchsorted(mid, mag, side="left")    # ties: the lower code ...
    hi = np.searchsorted(mid, mag, side="right")
    c = np.where((lo != hi) & (lo % 2 == 1), hi, lo)   # ... unless it is odd
    c = c + 128 * np.signbit(y)
    return np.where(np.isnan(y), 127, c), scale


def kv_inputs(rows, H, hd, dtype, seed, special=False):
    g = np.random.default_rng(seed)
    x = g.standard_normal((2, rows, H, hd)) * np.exp(3 * g.standard_normal((2, rows, H, 1)))
    t = torch.from_numpy(x).to(TD[dtype])
    if special and rows >= 8:
        t[:, 0] = 0
        t[0, 1, 0, 3], t[1, 1, 0, 5] = float("nan"), float("inf")
        t[0, 2, 0, :] = float("nan")
        t[0, 3, 0, :] = -float("inf")
        t[:, 4] = torch.finfo(TD[dtype]).max
        t[:, 5] = torch.finfo(TD[dtype]).smallest_normal
        t[:, 6, 0, 1:], t[:, 6, 0, 0] = 1.0, 448.0 * 64     # ties and codes below the grid
        t[:, 7, 0, :] = torch.arange(hd).to(TD[dtype]) / 16 - 3
    return t


def canonical(c):
    """All NaN codes as one."""
    return np.where((c & 127) == 127, 127, c)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("rows,H,hd,pos0,fused", [(1, 1, 64, 0, False), (1, 4, 128, 7, True), (9, 5, 64, 3, True),
                                                  (33, 8, 128, 0, False), (257, 3, 128, 11, True)])
def test_kv_quant_and_dequant(B, dtype, rows, H, hd, pos0, fused):
    """Codes, scales and read-back values equal the definition bit for bit; other rows stay."""
    t = kv_inputs(rows, H, hd, dtype, rows + H, special=True)
    if fused:      # slices of one projection's rows
        buf = torch.zeros(rows, 2 * H * hd + 16, dtype=TD[dtype])
        buf[:, :H * hd], buf[:, H * hd + 16:] = t[0].reshape(rows, -1), t[1].reshape(rows, -1)
        buf = buf.cuda()
        k, v = buf[:, :H * hd], buf[:, H * hd + 16:]
    else:
        k, v = (x.reshape(rows, -1).cuda() for x in t)
    cap = pos0 + rows + 5
    codes = torch.full((2, cap, H, hd), 0x5a, dtype=torch.uint8, device="cuda")
    scales = torch.full((2, H, cap), -7.0, device="cuda")
    B.op_kv_quant_async(k.data_ptr(), v.data_ptr(), code(B, dtype), k.stride(0), v.stride(0), rows, H, hd,
                        codes.data_ptr(), scales.data_ptr(), cap, pos0, stream())
    c, s = codes.cpu().numpy(), scales.cpu().numpy()
    rc, rs = quant_ref(t.double().numpy())
    p1 = pos0 + rows
    assert np.array_equal(canonical(c[:, pos0:p1]), canonical(rc))
    assert np.array_equal(s[:, :, pos0:p1], rs.transpose(0, 2, 1))
    assert (c[:, :pos0] == 0x5a).all() and (c[:, p1:] == 0x5a).all()
    assert (s[:, :, :pos0] == -7).all() and (s[:, :, p1:] == -7).all()
    # read back, into strided rows of every type
    for out in ("f16", "bf16", "f32"):
        y = torch.full((2, rows, H * hd + 8), 3.0, dtype=TD[out], device="cuda")
        B.op_kv_dequant_async(codes.data_ptr(), scales.data_ptr(), cap, pos0, rows, H, hd, y[0].data_ptr(),
                              y[1].data_ptr(), code(B, out), y.stride(1), y.stride(1), stream())
        top = torch.finfo(TD[out]).max
        ref = torch.from_numpy(E4M3[rc] * rs[..., None]).clamp(-top, top).float().to(TD[out])
        got = y[:, :, :H * hd].reshape(2, rows, H, hd).cpu()
        assert torch.equal(torch.nan_to_num(got.float(), nan=1e30), torch.nan_to_num(ref.float(), nan=1e30))
        assert (y[:, :, H * hd:] == 3.0).all()


@pytest.mark.parametrize("dtype", ["f16", "f32"])
def test_kv_unaligned_rows(B, dtype):
    """Rows that start off a 16-byte boundary (an odd stride, a shifted base) take the element
    loads and give the same."""
    rows, H, hd = 13, 2, 64
    t = kv_inputs(rows, H, hd, dtype, 5)
    buf = torch.zeros(2, rows, H * hd + 1, dtype=TD[dtype], device="cuda")
    buf[:, :, 1:] = t.reshape(2, rows, -1).cuda()
    k, v = buf[0, :, 1:], buf[1, :, 1:]
    codes = torch.zeros(2, rows, H, hd, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(2, H, rows, device="cuda")
    B.op_kv_quant_async(k.data_ptr(), v.data_ptr(), code(B, dtype), H * hd + 1, H * hd + 1, rows, H, hd,
                        codes.data_ptr(), scales.data_ptr(), rows, 0, stream())
    rc, rs = quant_ref(t.double().numpy())
    assert np.array_equal(codes.cpu().numpy(), rc) and np.array_equal(scales.cpu().numpy(), rs.transpose(0, 2, 1))
    back = torch.zeros_like(buf)
    B.op_kv_dequant_async(codes.data_ptr(), scales.data_ptr(), rows, 0, rows, H, hd, back[0, :, 1:].data_ptr(),
                          back[1, :, 1:].data_ptr(), code(B, dtype), H * hd + 1, H * hd + 1, stream())
    top = torch.finfo(TD[dtype]).max
    ref = torch.from_numpy(E4M3[rc] * rs[..., None]).clamp(-top, top).to(TD[dtype]).reshape(2, rows, -1)
    assert torch.equal(back[:, :, 1:].cpu(), ref) and (back[:, :, 0] == 0).all()


# ---- attention over a shared prefix ------------------------------------------------------------
def attn_ref(q, kp, vp, kn, vn, row0, lens, scale, out):
    """float64; kp, vp [P, Hkv, hd] (already the values used), kn None: prefix only."""
    Hq, Hkv = q.shape[1], kp.shape[1]
    for r0, n in zip(row0, lens):
        for i in range(n):
            for h in range(Hq):
                g = h * Hkv // Hq
                K = kp[:, g] if kn is None else np.concatenate([kp[:, g], kn[r0:r0 + i + 1, g]])
                V = vp[:, g] if kn is None else np.concatenate([vp[:, g], vn[r0:r0 + i + 1, g]])
                if len(K) == 0:
                    out[r0 + i, h] = 0
                    continue
                z = (K @ q[r0 + i, h]) * scale
                p = np.exp(z - z.max())
                out[r0 + i, h] = (p / p.sum()) @ V
    return out


class Attn:
    """Inputs of one call on the host (f16 values as float64) and on the device."""

    def __init__(self, B, Hq, Hkv, hd, P, lens, fmt="f16", gap=0, lead=0, tail=0, own=True, spread=1.0, seed=0):
        self.__dict__.update(B=B, Hq=Hq, Hkv=Hkv, hd=hd, P=P, lens=list(lens), fmt=fmt, own=own)
        self.row0, at = [], lead
        for n in lens:
            self.row0.append(at)
            at += n + gap
        self.R = R = max(1, at + tail)
        self.cap = cap = P + 9
        g = np.random.default_rng(seed + 31 * P + Hq + sum(lens))
        W = (Hq + 2 * Hkv) * hd
        x = torch.from_numpy(g.standard_normal((R, W)) * spread).half()
        self.x = x.cuda()
        kv = torch.from_numpy(g.standard_normal((2, cap, Hkv, hd)) * spread).half()
        kv[:, P:] = float("nan")                       # behind the prefix: never read
        self.scales = None
        if fmt == "f16":
            self.kv = kv.cuda()
            self.used = kv[:, :P].double().numpy()
        else:
            self.kv = torch.full((2, cap, Hkv, hd), 0x7f, dtype=torch.uint8, device="cuda")
            self.scales = torch.full((2, Hkv, cap), float("nan"), device="cuda")
            src = kv[:, :max(P, 1)].cuda().contiguous()
            if P:
                B.op_kv_quant_async(src[0].data_ptr(), src[1].data_ptr(), B.S1_F16, Hkv * hd, Hkv * hd, P, Hkv, hd,
                                    self.kv.data_ptr(), self.scales.data_ptr(), cap, 0, stream())
            v = E4M3[self.kv[:, :P].cpu().numpy()] * \
                self.scales[:, :, :P].cpu().numpy().astype(np.float64).transpose(0, 2, 1)[..., None]
            self.used = v.astype(np.float16).astype(np.float64)
        self.out = torch.full((R, Hq, hd), 55.0, dtype=torch.float16, device="cuda")
        self.scale = hd ** -0.5

    def parts(self):
        a, b = self.Hq * self.hd, (self.Hq + self.Hkv) * self.hd
        return self.x[:, :a], self.x[:, a:b], self.x[:, b:]

    def workspace(self):
        n = self.B.op_attention_shared_workspace(self.lens, self.P, self.Hq, self.Hkv, self.hd)
        return torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")

    def call(self, ws=None, st=None):
        q, k, v = self.parts()
        ws = self.workspace() if ws is None else ws
        self.ws = ws
        self.B.op_attention_shared_async(
            q.data_ptr(), q.stride(0), k.data_ptr() if self.own else 0, v.data_ptr() if self.own else 0, k.stride(0),
            self.row0, self.lens, self.kv.data_ptr() if self.P else 0,
            self.scales.data_ptr() if self.scales is not None else 0,
            self.B.S1_KV_F16 if self.fmt == "f16" else self.B.S1_KV_E4M3, self.P, self.cap, self.Hq, self.Hkv,
            self.hd, self.scale, self.out.data_ptr(), ws.data_ptr(), ws.numel(), stream() if st is None else st)

    def ref(self):
        q, k, v = (t.double().cpu().numpy().reshape(self.R, -1, self.hd) for t in self.parts())
        out = np.full((self.R, self.Hq, self.hd), 55.0)
        return attn_ref(q, self.used[0], self.used[1], k if self.own else None, v, self.row0, self.lens, self.scale,
                        out)

    def tol(self):
        """The weights are rounded to f16 (2^-11 each, so at most 2^-11 max |v| in a weighted mean)
        and so is the result (2^-11 of it); fp32 scores of at most a few hundred terms and exp move a
        weight by less than 2^-13 at these score sizes."""
        v = self.parts()[2].double().abs().max().item()
        if self.P:
            v = max(v, np.abs(self.used[1]).max())
        return (2 * 2.0 ** -11 + 2.0 ** -12) * v

    def check(self):
        self.call()
        self.B.op_sync(stream())
        got, ref = self.out.double().cpu().numpy(), self.ref()
        err = np.abs(got - ref).max()
        assert err <= self.tol(), (err, self.tol())
        live = np.zeros(self.R, bool)
        for r0, n in zip(self.row0, self.lens):
            live[r0:r0 + n] = True
        assert (got[~live] == 55).all()


SHAPES = [  # Hq, Hkv, hd, P, lens
    (1, 1, 64, 0, [1]), (4, 4, 128, 1, [1]), (16, 4, 128, 127, [1, 1, 1]), (16, 4, 128, 128, [3]),
    (40, 8, 128, 129, [1] * 7), (8, 2, 64, 255, [5, 33]), (6, 2, 128, 300, [200]), (12, 1, 64, 640, [9, 1, 30]),
    (4, 4, 64, 77, [129, 3]), (128, 1, 128, 200, [2, 1]), (64, 1, 64, 1030, [4]), (16, 4, 128, 1024, [48, 48, 48]),
    (40, 8, 128, 600, [64]), (4, 2, 128, 0, [130, 1, 40]), (10, 2, 64, 2500, [1, 0, 2, 0]), (3, 3, 64, 33, [0, 300, 0])]


@pytest.mark.parametrize("fmt", ["f16", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,hd,P,lens", SHAPES)
def test_attention_shared(B, Hq, Hkv, hd, P, lens, fmt):
    Attn(B, Hq, Hkv, hd, P, lens, fmt).check()


@pytest.mark.parametrize("fmt", ["f16", "e4m3"])
@pytest.mark.parametrize("P,lens,gap,lead,tail", [(200, [1] * 9, 7, 3, 5), (65, [40, 2, 90], 1, 0, 64),
                                                  (500, [16, 16, 16, 16], 48, 0, 48)])
def test_attention_padded_batch(B, P, lens, gap, lead, tail, fmt):
    """Rows between, before and behind the sequences hold NaN and infinities; they are not read
    into any result and their output rows stay as they were."""
    a = Attn(B, 8, 2, 128, P, lens, fmt, gap=gap, lead=lead, tail=tail)
    dead = torch.ones(a.R, dtype=torch.bool)
    for r0, n in zip(a.row0, a.lens):
        dead[r0:r0 + n] = False
    idx = dead.nonzero()[:, 0].cuda()
    a.x[idx] = torch.where(torch.arange(a.x.shape[1], device="cuda") % 2 == 0, float("nan"), float("inf")).half()
    a_ref = a.x.clone()
    a.x[idx] = 0
    ref = a.ref()
    a.x = a_ref
    a.call()
    got = a.out.double().cpu().numpy()
    assert np.abs(got - ref).max() <= (2 * 2.0 ** -11 + 2.0 ** -12) * 6
    assert (got[dead.numpy()] == 55).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("where", ["k", "v", "q"])
def test_attention_isolates_sequences(B, bad, where):
    """A non-finite value in one sequence's row reaches that sequence's rows from there on and
    nothing else, as the formula has it."""
    lens = [5, 9, 1, 12]
    a = Attn(B, 8, 2, 64, 150, lens)
    clean = a.ref()
    r = a.row0[1] + 4                                # row 4 of sequence 1
    part = a.parts()[{"q": 0, "k": 1, "v": 2}[where]]
    part[r, 5] = bad                                 # head 0 of kv (or q) heads
    a.call()
    got = a.out.double().cpu().numpy()
    seen = np.zeros((a.R, 8), bool)
    if where == "q":
        seen[r, 0] = True
    else:
        seen[r:a.row0[1] + 9, :4] = True             # q heads of kv head 0
    tol = a.tol() if math.isfinite(a.tol()) else (2 * 2.0 ** -11 + 2.0 ** -12) * 6
    ok = np.abs(got - clean) <= tol
    assert ok[~seen].all()
    if where == "v":
        hit = np.zeros(64, bool)
        hit[5] = True
        assert ok[seen][:, ~hit].all()
        v = got[seen][:, 5]
        assert np.isnan(v).all() if math.isnan(bad) else (v == bad).all()
    elif math.isnan(bad) or where == "q":
        assert np.isnan(got[seen]).all()
    else:      # an infinite key: a score of +inf (NaN result) or -inf (the key drops out)
        assert (np.isnan(got[seen]).all(-1) | np.isfinite(got[seen]).all(-1)).all()


def test_attention_nan_in_the_prefix(B):
    """Every row sees the whole prefix: a NaN there is in every row's result, in its column (v) or
    wholly (k), for the q heads of that kv head."""
    a = Attn(B, 4, 2, 64, 300, [3, 2])
    a.kv[1, 257, 0, 9] = float("nan")
    clean = a.ref()
    a.call()
    got = a.out.double().cpu().numpy()
    col = np.arange(64) == 9
    assert np.isnan(got[:, :2, 9]).all()
    ok = np.abs(got - clean) <= a.tol()
    assert ok[:, :2][:, :, ~col].all() and ok[:, 2:].all()


@pytest.mark.parametrize("fmt", ["f16", "e4m3"])
def test_attention_prefix_only(B, fmt):
    """No own rows: queries see the prefix; with an empty prefix as well the result is zero."""
    Attn(B, 8, 2, 128, 300, [3, 1, 20], fmt, own=False).check()
    Attn(B, 8, 2, 128, 0, [3, 1], fmt, own=False).check()


@pytest.mark.parametrize("fmt", ["f16", "e4m3"])
def test_attention_growing_maxima(B, fmt):
    """Scores that rise along the prefix by hundreds: the running maximum moves in every tile."""
    a = Attn(B, 4, 1, 64, 1000, [2, 3], fmt)
    u = torch.ones(64)
    k = (torch.linspace(-4, 9, 1000)[:, None] * u).half()
    if fmt == "f16":
        a.kv[0, :1000, 0] = k.cuda()
        a.used[0][:, 0] = k.double().numpy()
    else:
        c, s = quant_ref(k.double().numpy())
        a.kv[0, :1000, 0] = torch.from_numpy(c.astype(np.uint8)).cuda()
        a.scales[0, 0, :1000] = torch.from_numpy(s).float().cuda()
        a.used[0][:, 0] = (E4M3[c] * s[:, None])
    a.x[:, :4 * 64] = 1.5
    # scores reach 1.5 * 9 * 8 = 108: fp32 sums of 64 terms are off by less than 64 * 2^-24 * 108,
    # which moves a weight by less than 2^-11 more
    a.call()
    err = np.abs(a.out.double().cpu().numpy() - a.ref()).max()
    assert err <= 3.5 * 2.0 ** -11 * max(np.abs(a.used[1]).max(), 6)


def test_attention_snapshot_scales_out_of_the_ordinary(B):
    """8-bit rows whose scale is far from 1: read back as the f16 the read-back gives (held at the
    largest f16, flushed below the smallest)."""
    a = Attn(B, 2, 1, 64, 40, [2], "e4m3", spread=0.05)
    g = np.random.default_rng(3)
    c = g.integers(0, 126, (2, 40, 64)).astype(np.uint8)
    E = np.concatenate([np.arange(-30, -10), np.arange(-12, 8)])
    E[0], E[1], E[-1] = -126, -33, 9
    sc = np.stack([2.0 ** np.minimum(E, -7), 2.0 ** E])           # (small keys: even weights)
    a.kv[:, :40, 0] = torch.from_numpy(c).cuda()
    a.scales[:, 0, :40] = torch.from_numpy(sc).float().cuda()
    v = np.clip(E4M3[c] * sc[..., None], -65504, 65504)
    a.used = v.astype(np.float16).astype(np.float64)[:, :, None]
    a.check()


@pytest.mark.parametrize("n", [65, 300, 2300])
def test_attention_many_sequences(B, n):
    """More sequences than one launch's small and large tables hold."""
    lens = [(1, 0, 2, 1)[i % 4] for i in range(n)]
    Attn(B, 2, 1, 64, 20, lens).check()


@pytest.mark.parametrize("fmt", ["f16", "e4m3"])
def test_attention_long_prefix_splits(B, fmt):
    """A long prefix for few rows is split over many CTAs and joined; the join is in a fixed order,
    so results repeat bit for bit, and a workspace's earlier contents do not matter."""
    a = Attn(B, 8, 2, 128, 20011, [1, 3], fmt)
    ws = a.workspace()
    ws.fill_(0xff)
    a.call(ws)
    first = a.out.clone()
    ws.fill_(0x3c)
    a.out.fill_(55)
    a.call(ws)
    assert torch.equal(first, a.out)
    assert np.abs(first.double().cpu().numpy() - a.ref()).max() <= a.tol()


@pytest.mark.parametrize("fmt", ["f16", "e4m3"])
def test_attention_graph_and_side_stream(B, fmt):
    """Captured once and replayed on new contents of the same buffers, on a side stream."""
    a = Attn(B, 16, 4, 128, 3000, [1] * 5, fmt)
    b = Attn(B, 16, 4, 128, 3000, [1] * 5, fmt, seed=9)
    ws = a.workspace()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        a.call(ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            a.call(ws)
        a.out.fill_(55)
        g.replay()
        one = a.out.clone()
        for dst, src in ((a.x, b.x), (a.kv, b.kv)) + (((a.scales, b.scales),) if a.scales is not None else ()):
            dst.copy_(src)
        a.out.fill_(55)
        g.replay()
        two = a.out.clone()
    st.synchronize()
    assert np.abs(two.double().cpu().numpy() - b.ref()).max() <= b.tol()
    c = Attn(B, 16, 4, 128, 3000, [1] * 5, fmt)
    assert np.abs(one.double().cpu().numpy() - c.ref()).max() <= c.tol()


# ---- linear attention ----------------------------------------------------------------------------
def lin_ref(q, k, v, lam, scale, S0, rows):
    """float64 recurrence over one sequence's rows; returns outputs and the final state, and the same
    with every factor's magnitude (what roundings of the terms can be charged against)."""
    S, A = S0.copy(), np.abs(S0)
    o, oa = [], []
    for t in rows:
        S = lam[:, None, None] * S + v[t][:, :, None] * k[t][:, None, :]
        A = lam[:, None, None] * A + np.abs(v[t][:, :, None] * k[t][:, None, :])
        o.append(scale * np.einsum("hij,hj->hi", S, q[t]))
        oa.append(scale * np.einsum("hij,hj->hi", A, np.abs(q[t])))
    H, dv = v.shape[1], v.shape[2]
    return np.array(o).reshape(-1, H, dv), S, np.array(oa).reshape(-1, H, dv), A


class Lin:
    def __init__(self, B, H, dk, dv, lens, dtype, state="none", keep=True, gap=0, lead=0, tail=0, seed=0, mag=1.0,
                 log_decay=None):
        self.__dict__.update(B=B, H=H, dk=dk, dv=dv, lens=list(lens), dtype=dtype, state=state, keep=keep)
        self.row0, at = [], lead
        for n in lens:
            self.row0.append(at)
            at += n + gap
        self.R = R = max(1, at + tail)
        self.n = n = len(lens)
        g = np.random.default_rng(seed + 7 * H + dk + dv + sum(lens))
        x = torch.from_numpy(g.standard_normal((R, H * (2 * dk + dv))) * mag).to(TD[dtype])
        self.x = x.cuda()
        ld = -2.0 ** (-8.0 * np.arange(1, H + 1) / H) if log_decay is None else np.asarray(log_decay, np.float64)
        self.ld = torch.from_numpy(ld).float().cuda()
        self.per = H * dk * dv
        m = {"none": 0, "shared": 1, "own": n}[state]
        self.S_in = torch.from_numpy(g.standard_normal((m, H, dv, dk)) * 2 * mag).float().cuda() if m else None
        self.S_out = torch.full((n, H, dv, dk), 9.0, device="cuda") if keep else None
        self.out = torch.full((R, H, dv), 55.0, dtype=TD[dtype], device="cuda")
        self.scale = dk ** -0.5

    def parts(self):
        a, b = self.H * self.dk, 2 * self.H * self.dk
        return self.x[:, :a], self.x[:, a:b], self.x[:, b:]

    def args(self):
        q, k, v = self.parts()
        return (q.data_ptr(), k.data_ptr(), v.data_ptr(), code(self.B, self.dtype), q.stride(0), k.stride(0),
                v.stride(0), self.ld.data_ptr())

    def states(self):
        s_in = self.S_in.data_ptr() if self.S_in is not None else 0
        return s_in, self.per if self.state == "own" else 0, self.S_out.data_ptr() if self.S_out is not None else 0

    def call(self, ws=None, st=None):
        if ws is None:
            n = self.B.op_linattn_workspace(self.lens, self.H, self.dk, self.dv)
            ws = torch.full((max(n, 16),), 0xff, dtype=torch.uint8, device="cuda")
        self.ws = ws
        self.B.op_linattn_async(*self.args(), self.row0, self.lens, self.H, self.dk, self.dv, self.scale,
                                *self.states(), self.out.data_ptr(), ws.data_ptr(), ws.numel(),
                                stream() if st is None else st)

    def step(self):
        self.B.op_linattn_step_async(*self.args(), self.n, self.H, self.dk, self.dv, self.scale, *self.states(),
                                     self.out.data_ptr(), stream())

    def ref(self):
        q, k, v = (t.double().cpu().numpy().reshape(self.R, self.H, -1) for t in self.parts())
        lam = np.exp(np.minimum(self.ld.double().cpu().numpy(), 0))
        out = np.full((self.R, self.H, self.dv), 55.0)
        mag = np.zeros_like(out)
        Ss, As = [], []
        for s, (r0, n) in enumerate(zip(self.row0, self.lens)):
            S0 = np.zeros((self.H, self.dv, self.dk))
            if self.S_in is not None:
                S0 = self.S_in[s if self.state == "own" else 0].double().cpu().numpy()
            o, S, oa, A = lin_ref(q, k, v, lam, self.scale, S0, range(r0, r0 + n))
            out[r0:r0 + n], mag[r0:r0 + n] = o, oa
            Ss.append(S)
            As.append(A)
        return out, mag, np.array(Ss), np.array(As)

    def compare(self):
        """Outputs: the weights within a chunk, the state, and the result are each rounded once to the
        rows' type (u each, against the sum of magnitudes; the state's operand form only ever for
        products), and decays of fp32 logs are off by less than 2^-20. States: fp32 sums of products
        whose factors carry at least 16 bits (2^-17 each)."""
        out, mag, S, A = self.ref()
        got = self.out.double().cpu().numpy()
        u = U[self.dtype]
        err = np.abs(got - out)
        assert (err <= 3 * u * mag + 1e-6 * mag + 1e-7).all(), (err.max(), (err / (mag + 1e-30)).max() / u)
        live = np.zeros(self.R, bool)
        for r0, n in zip(self.row0, self.lens):
            live[r0:r0 + n] = True
        assert (got[~live] == 55).all()
        if self.keep:
            es = np.abs(self.S_out.double().cpu().numpy() - S)
            assert (es <= (2.0 ** -16 + 2.0 ** -18) * A + 1e-9).all(), (es / (A + 1e-30)).max()

    def check(self):
        self.call()
        self.B.op_sync(stream())
        self.compare()


LIN = [  # H, dk, dv, lens, state
    (1, 64, 64, [1], "none"), (2, 128, 128, [2], "own"), (3, 128, 64, [63, 1, 64], "shared"),
    (2, 64, 128, [65, 0, 127], "own"), (4, 128, 128, [128, 129], "none"), (1, 128, 128, [700], "own"),
    (2, 64, 64, [333, 5, 0, 1, 200], "shared"), (5, 128, 128, [31, 300], "own"), (1, 64, 128, [2100], "none")]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("H,dk,dv,lens,state", LIN)
def test_linattn(B, H, dk, dv, lens, state, dtype):
    Lin(B, H, dk, dv, lens, dtype, state).check()


def test_linattn_without_final_states(B):
    Lin(B, 2, 128, 128, [200, 3], "f16", "own", keep=False).check()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_linattn_decays(B, dtype):
    """No decay, almost none, one token's memory, none at all (-inf), and a positive log taken as 0."""
    Lin(B, 6, 64, 64, [150, 70], dtype, "own", log_decay=[0.0, -1e-4, -3.0, -90.0, -np.inf, 0.5]).check()


@pytest.mark.parametrize("mag", [1e-2, 30.0])
def test_linattn_magnitudes(B, mag):
    """Products far above f16's range and states far below its normal range keep their precision
    (k and v of 1e-2 make states of 1e-4; q.k of 30^2 * 64 is above 65504 before the scale)."""
    a = Lin(B, 2, 64, 64, [140], "bf16", "own", mag=mag)
    a.check()
    b = Lin(B, 2, 64, 64, [140], "f16", "own", mag=mag)
    b.scale = 1e-3 if mag > 1 else 1.0              # (outputs within f16)
    b.check()


@pytest.mark.parametrize("gap,lead,tail", [(5, 2, 9), (70, 0, 64)])
def test_linattn_padded_batch(B, gap, lead, tail):
    """Unused rows hold NaN and are neither read into results nor written."""
    a = Lin(B, 2, 128, 64, [40, 64, 1, 100], "f16", "shared", gap=gap, lead=lead, tail=tail)
    dead = torch.ones(a.R, dtype=torch.bool)
    for r0, n in zip(a.row0, a.lens):
        dead[r0:r0 + n] = False
    a.x[dead.nonzero()[:, 0].cuda()] = float("nan")
    a.check()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("which", [0, 1, 2])
def test_linattn_nonfinite_rows(B, bad, which):
    """A non-finite value reaches its own row (q) or rows from its own on (k, v), never an earlier
    row, another head, or another sequence."""
    a = Lin(B, 2, 64, 64, [50, 140], "f16", "none", keep=True)
    b = Lin(B, 2, 64, 64, [50, 140], "f16", "none", keep=True)
    b.check()
    t = 50 + 70
    a.parts()[which][t, 3] = bad                     # head 0
    a.call()
    got, ref = a.out.double().cpu().numpy(), b.out.double().cpu().numpy()
    assert np.array_equal(got[:t], ref[:t]) and np.array_equal(got[:, 1], ref[:, 1])
    So, Sr = a.S_out.cpu().numpy(), b.S_out.cpu().numpy()
    assert np.array_equal(So[0], Sr[0]) and np.array_equal(So[1, 1], Sr[1, 1])
    if which == 0:
        assert not np.isfinite(got[t, 0]).any() and np.array_equal(got[t + 1:], ref[t + 1:])
        assert np.array_equal(So, Sr)
    elif which == 1:     # column 3 of the state
        assert not np.isfinite(got[t:, 0]).any()
        assert not np.isfinite(So[1, 0][:, 3]).any() and np.isfinite(So[1, 0][:, 4:]).all()
    else:                # row 3 of the state, column 3 of the outputs
        assert not np.isfinite(got[t:, 0, 3]).any() and np.array_equal(got[:, 0, 4:], ref[:, 0, 4:])
        assert not np.isfinite(So[1, 0, 3]).any() and np.isfinite(So[1, 0, 4:]).all()


def test_linattn_in_place_and_in_parts(B):
    """A prompt in two calls, states advanced in place, against one call."""
    one = Lin(B, 2, 128, 128, [300, 90], "bf16", "own")
    one.call()
    two = Lin(B, 2, 128, 128, [300, 90], "bf16", "own")
    two.S_out = two.S_in
    two.row0, two.lens = [0, 300], [130, 1]
    two.call()
    two.row0, two.lens = [130, 301], [170, 89]
    two.call()
    out, mag, S, A = one.ref()
    assert (np.abs(two.out.double().cpu().numpy() - out) <= 3 * U["bf16"] * mag + 1e-6 * mag).all()
    assert (np.abs(two.S_in.double().cpu().numpy() - S) <= 2.0 ** -15 * A).all()


@pytest.mark.parametrize("n", [65, 2100])
def test_linattn_many_sequences(B, n):
    Lin(B, 1, 64, 64, [(1, 0, 3)[i % 3] for i in range(n)], "f16", "shared").check()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("H,dk,dv,n,state,keep", [(1, 64, 64, 1, "none", True), (3, 128, 128, 5, "own", True),
                                                  (2, 64, 128, 7, "shared", False), (4, 128, 64, 300, "shared", True),
                                                  (16, 128, 128, 3, "shared", False)])
def test_linattn_step(B, H, dk, dv, n, state, keep, dtype):
    a = Lin(B, H, dk, dv, [1] * n, dtype, state, keep)
    a.step()
    a.compare()


def test_linattn_step_in_place(B):
    """Tokens one by one, states advanced in place, against the prompt form over the same rows."""
    H, D, n, T = 2, 128, 3, 5
    a = Lin(B, H, D, D, [T] * n, "f16", "own")
    a.call()
    S = a.S_in.clone()
    rows = torch.zeros(n, a.x.shape[1], dtype=torch.float16, device="cuda")
    o = torch.zeros(n, H, D, dtype=torch.float16, device="cuda")
    for t in range(T):
        rows.copy_(a.x[t::T])
        q, k, v = rows[:, :H * D], rows[:, H * D:2 * H * D], rows[:, 2 * H * D:]
        B.op_linattn_step_async(q.data_ptr(), k.data_ptr(), v.data_ptr(), B.S1_F16, rows.stride(0), rows.stride(0),
                                rows.stride(0), a.ld.data_ptr(), n, H, D, D, a.scale, S.data_ptr(), a.per,
                                S.data_ptr(), o.data_ptr(), stream())
        out, mag, _, _ = a.ref()
        err = np.abs(o.double().cpu().numpy() - out[t::T])
        assert (err <= 3 * U["f16"] * mag[t::T] + 1e-6).all()
    assert torch.allclose(S, a.S_out, rtol=1e-4, atol=1e-4)


def test_linattn_graph(B):
    a = Lin(B, 2, 128, 128, [500, 20], "f16", "own")
    ws = torch.empty(max(16, B.op_linattn_workspace(a.lens, 2, 128, 128)), dtype=torch.uint8, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        a.call(ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            a.call(ws)
        b = Lin(B, 2, 128, 128, [500, 20], "f16", "own", seed=4)
        a.x.copy_(b.x)
        a.S_in.copy_(b.S_in)
        g.replay()
    st.synchronize()
    a.compare()


# ---- together, as they are used --------------------------------------------------------------------
def test_prefix_snapshot_and_questions(B):
    """One prefix, written once (8-bit K/V, linear state), then a batch of questions and a round of
    single tokens continuing it, on one stream without a synchronisation in between."""
    P, lens, Hq, Hkv, hd = 700, [5, 1, 12], 8, 2, 64
    a = Attn(B, Hq, Hkv, hd, P, lens, "e4m3")
    rows = Lin(B, 4, 64, 64, [P], "f16", "none")                  # the linear layer's prefix
    rows.call()
    qs = Lin(B, 4, 64, 64, lens, "f16", "shared", keep=True, seed=3)
    qs.S_in = rows.S_out
    qs.call()
    a.call()
    tok = Lin(B, 4, 64, 64, [1, 1, 1], "f16", "own", keep=True, seed=5)
    tok.S_in = qs.S_out
    tok.step()
    B.op_sync(stream())
    assert np.abs(a.out.double().cpu().numpy() - a.ref()).max() <= a.tol()
    rows.compare()
    qs.compare()
    tok.compare()


# ---- what a caller may do besides ------------------------------------------------------------------
@pytest.mark.parametrize("fmt", ["f16", "e4m3"])
def test_snapshot_offsets_past_32_bits(B, fmt):
    """Rows whose byte offset in a plane lies past 2^32: written and read back (e4m3), and attended to.
    The other 2^26 (2^25) rows are zeros: five keys score 64 above them, so those weigh e^-64 each
    (2^26 of them less than 2^-60), and the five equally: the result is the mean of five values,
    after the weights (exactly 1) rounded once to f16, with fp32 sums: 2^-11 of the largest value."""
    hd, n = 64, 5
    cap = (1 << 26 if fmt == "e4m3" else 1 << 25) + 1000
    g = np.random.default_rng(5)
    k = torch.full((n, hd), 2.0, dtype=torch.float16, device="cuda")
    v = torch.from_numpy(g.standard_normal((n, hd))).half().cuda()
    if fmt == "e4m3":
        kv = torch.zeros(2, cap, 1, hd, dtype=torch.uint8, device="cuda")
        scales = torch.ones(2, 1, cap, device="cuda")
        B.op_kv_quant_async(k.data_ptr(), v.data_ptr(), B.S1_F16, hd, hd, n, 1, hd, kv.data_ptr(), scales.data_ptr(),
                            cap, cap - n, stream())
        c, sc = quant_ref(v.double().cpu().numpy())
        used = E4M3[c] * sc[:, None]
        assert np.array_equal(kv[1, cap - n:, 0].cpu().numpy(), c)
        assert not kv[:, :cap - n].any()
        back = torch.full((2, n, hd), 7.0, dtype=torch.float16, device="cuda")
        B.op_kv_dequant_async(kv.data_ptr(), scales.data_ptr(), cap, cap - n, n, 1, hd, back[0].data_ptr(),
                              back[1].data_ptr(), B.S1_F16, hd, hd, stream())
        assert np.array_equal(back[1].double().cpu().numpy(), used) and (back[0] == 2).all()
    else:
        kv = torch.zeros(2, cap, 1, hd, dtype=torch.float16, device="cuda")
        kv[0, cap - n:, 0], kv[1, cap - n:, 0] = k, v
        scales, used = None, v.double().cpu().numpy()
    q = torch.ones(1, 1, hd, dtype=torch.float16, device="cuda")
    out = torch.full((1, 1, hd), 55.0, dtype=torch.float16, device="cuda")
    nb = B.op_attention_shared_workspace([1], cap, 1, 1, hd)
    ws = torch.empty(max(nb, 16), dtype=torch.uint8, device="cuda")
    B.op_attention_shared_async(q.data_ptr(), hd, 0, 0, 0, [0], [1], kv.data_ptr(),
                                0 if scales is None else scales.data_ptr(),
                                B.S1_KV_F16 if fmt == "f16" else B.S1_KV_E4M3, cap, cap, 1, 1, hd, 0.5, out.data_ptr(),
                                ws.data_ptr(), ws.numel(), stream())
    B.op_sync(stream())
    err = np.abs(out[0, 0].double().cpu().numpy() - used.mean(0)).max()
    assert err <= 2.0 ** -11 * np.abs(used).max() + 1e-7, err


@pytest.mark.parametrize("graphs", [False, True])
def test_calls_at_once(B, graphs):
    """Calls on two streams, eager or replayed, each with buffers and a workspace of its own: the bits
    of the calls made alone."""
    ops = [Attn(B, 16, 4, 128, 5000, [3, 1], "e4m3"), Attn(B, 16, 4, 128, 5000, [40, 1, 200], "f16"),
           Lin(B, 4, 128, 128, [900, 20], "bf16", "own"), Lin(B, 4, 128, 128, [300] * 3, "f16", "shared")]
    alone = []
    for a in ops:
        a.call()
        B.op_sync(stream())
        alone.append((a.out.clone(), a.S_out.clone() if isinstance(a, Lin) else None))
        a.out.fill_(55)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    pairs = [(ops[i], streams[i % 2]) for i in range(4)]
    held = {}
    if graphs:
        for i, (a, st) in enumerate(pairs):
            with torch.cuda.stream(st):
                held[i] = torch.cuda.CUDAGraph()
                with torch.cuda.graph(held[i], stream=st):
                    a.call(a.ws)
        torch.cuda.synchronize()
    for _ in range(8):
        for i, (a, st) in enumerate(pairs):
            with torch.cuda.stream(st):
                held[i].replay() if graphs else a.call(a.ws, st.cuda_stream)
    for st in streams:
        B.op_sync(st.cuda_stream)
    for a, (out, S) in zip(ops, alone):
        assert torch.equal(a.out, out)
        assert S is None or torch.equal(a.S_out, S)


def test_short_calls_behind_a_long_one(B):
    """Calls are launched while the one before still runs; none starts before its end or gives up on it."""
    long = Attn(B, 16, 4, 128, 3000, [700] * 6, "f16")
    short = Attn(B, 16, 4, 128, 257, [2, 1], "e4m3")
    for a in (long, short):
        a.call()
    torch.cuda.synchronize()
    one, two = long.out.clone(), short.out.clone()
    for _ in range(5):
        long.out.fill_(55)
        short.out.fill_(55)
        for a in (long, short, long, short, short):
            a.call(a.ws)
    B.op_sync(stream())
    assert torch.equal(one, long.out) and torch.equal(two, short.out)
    assert np.abs(two.double().cpu().numpy() - short.ref()).max() <= short.tol()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("lens", [[2, 3], [130, 128], [300]])
def test_linattn_states_keep_fp32(B, dtype, lens):
    """Rounded factors would show in the returned states: two bf16 parts of a decayed value leave up to
    2^-18 of it. Parts leave at most 2^-24; fp32 decays of up to 300 rows (the log and its exponential
    2^-23 each, once a row in the reference's terms and once a chunk here) and sums of 2^-24 a step stay
    below 2^-20."""
    a = Lin(B, 3, 128, 64, lens, dtype, "own", log_decay=[-0.01, -0.3, -0.0005])
    a.call()
    B.op_sync(stream())
    _, _, S, A = a.ref()
    es = np.abs(a.S_out.double().cpu().numpy() - S)
    assert (es <= 2.0 ** -20 * A).all(), (es / (A + 1e-30)).max()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_linattn_outputs_of_a_long_memory(B, dtype):
    """Outputs that come from the state alone (zero keys after it): Q and its decay take no rounding of
    their own, so the error is the state's copy and the result, half a step each, and fp32's."""
    a = Lin(B, 2, 128, 128, [100], dtype, "own", log_decay=[-0.004, -0.05])
    q, k, v = a.parts()
    k.zero_()
    a.call()
    B.op_sync(stream())
    out, _, _, _ = a.ref()
    qd = np.abs(q.double().cpu().numpy().reshape(100, 2, 128))
    S0 = np.abs(a.S_in.double().cpu().numpy()[0])
    lam = np.exp(a.ld.double().cpu().numpy())
    mag = a.scale * np.einsum("hij,thj->thi", S0, qd) * lam[None, :, None] ** np.arange(1, 101)[:, None, None]
    u = U[dtype]
    err = np.abs(a.out.double().cpu().numpy() - out)
    assert (err <= u * mag + u * np.abs(out) + 2.0 ** -18 * mag).all(), (err / (mag + 1e-30)).max() / u


class LongLin(Lin):
    """As Lin, with the recurrence in 64 bits on the GPU (all heads of a row at once), for thousands of rows."""

    def ref(self):
        q, k, v = (t.double().reshape(self.R, self.H, -1) for t in self.parts())
        lam = torch.exp(self.ld.double().clamp(max=0))[:, None, None]
        out = torch.full((self.R, self.H, self.dv), 55.0, dtype=torch.float64, device="cuda")
        mag = torch.zeros_like(out)
        Ss, As = [], []
        for s, (r0, n) in enumerate(zip(self.row0, self.lens)):
            S = torch.zeros(self.H, self.dv, self.dk, dtype=torch.float64, device="cuda")
            if self.S_in is not None:
                S = self.S_in[s if self.state == "own" else 0].double()
            A = S.abs()
            for t in range(r0, r0 + n):
                x = v[t][:, :, None] * k[t][:, None, :]
                S, A = lam * S + x, lam * A + x.abs()
                out[t] = self.scale * (S @ q[t][:, :, None])[..., 0]
                mag[t] = self.scale * (A @ q[t].abs()[:, :, None])[..., 0]
            Ss.append(S)
            As.append(A)
        return tuple(x.cpu().numpy() for x in (out, mag, torch.stack(Ss), torch.stack(As)))


@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 128)])
def test_linattn_f16_many_chunks_at_full_load(B, dk, dv):
    """Every SM works through many f16 chunks whose magnitudes differ by 2^12 (keys and values by 2^6 each
    from one chunk to the next, queries with a period of three): each chunk's scales are its own. Against the
    recurrence (compare()'s tolerance), and the same bits 50 times, alone and beside a call on another stream."""
    lens = [2900, 2817, 3000, 2560, 2700]
    a = LongLin(B, 32, dk, dv, lens, "f16", "own")
    q, k, v = a.parts()
    for r0, n in zip(a.row0, a.lens):
        c = torch.arange(n, device="cuda") // 128
        loud = torch.where(c % 2 == 0, 8.0, 0.125).half()[:, None]
        k[r0:r0 + n] *= loud
        v[r0:r0 + n] *= loud
        q[r0:r0 + n] *= (2.0 ** (-2.0 * (c % 3))).half()[:, None]
    a.check()
    one, S = a.out.clone(), a.S_out.clone()
    b = Lin(B, 32, dk, dv, [1500, 1400, 1300], "f16", "shared", seed=2)
    b.call()
    torch.cuda.synchronize()
    b_one = b.out.clone()
    other = torch.cuda.Stream()
    for i in range(50):
        a.out.fill_(55)
        a.S_out.fill_(9)
        if i >= 25:
            b.call(b.ws, other.cuda_stream)
        a.call(a.ws)
        assert torch.equal(a.out, one) and torch.equal(a.S_out, S), i
    B.op_sync(other.cuda_stream)
    B.op_sync(stream())
    assert torch.equal(b.out, b_one)


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("P", [1, 33, 100, 129, 1000])
def test_attention_snapshot_without_spare_rows(B, P, hd):
    """An 8-bit snapshot of exactly P rows, codes and scales each the whole of their allocation, whose
    last key tile is not full."""
    a = Attn(B, 4, 2, hd, P, [3, 1], "e4m3")
    a.kv, a.scales, a.cap = a.kv[:, :P].contiguous(), a.scales[:, :, :P].contiguous(), P
    a.check()


def _outlier_call(B, which, value, lens, state, dtype, log_decay):
    a = Lin(B, 2, 128, 128, lens, dtype, state, log_decay=log_decay, seed=11)
    a.scale = 2.0 ** -10                 # (outputs of the outlier's own rows within f16)
    if value is not None:
        if which == "S":
            a.S_in[-1, 0, 7, 9] = value
        else:
            a.parts()["qkv".index(which)][a.row0[1] + which_row(which), 5] = value
    return a


def which_row(which):
    return 31 if which in "qv" else 127


@pytest.mark.parametrize("log_decay", [[-0.01, -0.01], [-1.5, -0.01], [-0.0005, -0.3]])
@pytest.mark.parametrize("state", ["none", "own"])
@pytest.mark.parametrize("value", [256.0, 4000.0, 60000.0])
@pytest.mark.parametrize("which", ["q", "k", "v", "S"])
def test_linattn_f16_outliers(B, which, value, state, log_decay):
    """One large finite element (row 31 or 127 of the second sequence, or of its initial state): the rows
    that do not see it keep their bits, those that do keep compare()'s tolerance (their sums of magnitudes
    hold the large terms only where the formula has them)."""
    if which == "S" and state == "none":
        pytest.skip("no initial state")
    lens = [40, 300]
    a = _outlier_call(B, which, value, lens, state, "f16", log_decay)
    b = _outlier_call(B, which, None, lens, state, "f16", log_decay)
    a.check()
    b.check()
    first = 0 if which == "S" else a.row0[1] + which_row(which)
    assert torch.equal(a.out[:40], b.out[:40]) and torch.equal(a.out[:, 1], b.out[:, 1])
    assert torch.equal(a.out[:max(first, 40)], b.out[:max(first, 40)])
    assert torch.equal(a.S_out[0], b.S_out[0])
    if which == "q":
        assert torch.equal(a.out[first + 1:], b.out[first + 1:]) and torch.equal(a.S_out, b.S_out)


@pytest.mark.parametrize("fmt", ["f16", "e4m3"])
@pytest.mark.parametrize("gap", [12.0, 16.0, 17.0, 18.0])
@pytest.mark.parametrize("where", [0, 65535, 30001])
def test_attention_sink(B, fmt, gap, where):
    """One key scores `gap` above 65535 equal others and has the value zero (an attention sink): the result is
    the others' mean value times their share of the weights. Their weights are equal, so each is rounded to f16
    alike: by half a step, 2^-11, where e^-gap >= 2^-24, else by 2^-35 of the sink's weight; the result's own
    rounding is 2^-11 of it. fp32 scores and exponentials are off by less than 2^-18, and the tensor cores' sums of
    at most 4096 steps, each dropping less than 2^-23 of the sum so far, by less than 2^-12."""
    hd, P = 64, 65536
    g = np.random.default_rng(4)
    v = torch.from_numpy(1 + 0.25 * g.random((P, hd))).half()
    v[where] = 0
    k = torch.zeros(P, hd).half()
    k[where] = 2                             # scale 1 / 8, q = gap / 16: score 64 * 2 * gap / 128
    a = Attn(B, 1, 1, hd, P, [1], fmt, own=False)
    a.x[:] = gap / 16
    src = torch.stack([k, v]).cuda().contiguous()
    if fmt == "f16":
        a.kv[:, :P, 0] = src
        used = v.double().numpy()
    else:
        B.op_kv_quant_async(src[0].data_ptr(), src[1].data_ptr(), B.S1_F16, hd, hd, P, 1, hd, a.kv.data_ptr(),
                            a.scales.data_ptr(), a.cap, 0, stream())
        used = E4M3[a.kv[1, :P, 0].cpu().numpy()] * a.scales[1, 0, :P].double().cpu().numpy()[:, None]
    ref = used.sum(0) / (P - 1 + math.exp(gap))
    a.call()
    B.op_sync(stream())
    err = np.abs(a.out[0, 0].double().cpu().numpy() - ref) / ref
    assert err.max() <= max(2.0 ** -11, 2.0 ** -35 * math.exp(gap)) + 2.0 ** -11 + 2.0 ** -12 + 2.0 ** -18, err.max()


def test_attention_sink_first_of_a_million(B):
    """A sink 17 above the 2^20 - 1 keys behind it, for so many rows that their sums need no split over CTAs: the
    small weights (2^-24.5 of the sink's) together weigh 4 percent, and reach the sum although each alone is below
    half of its last bit. A half tile's 32 terms a lane are exact to 2^-19 and together 11.07 steps (2^-13) of a
    sum of 2^10, so at least 11 are added: 0.7 percent of those 4, 2^-11 of the sum. Else as in
    test_attention_sink, with 2^-8 for the products' sums."""
    hd, P, Hq, rows, gap = 64, 1 << 20, 4, 9728, 17.0
    g = np.random.default_rng(4)
    v = torch.from_numpy(1 + 0.25 * g.random((P, hd))).half().cuda()
    v[0] = 0
    a = Attn(B, Hq, 1, hd, P, [rows], "f16", own=False)
    a.x[:] = gap / 16
    a.kv[0, :P] = 0
    a.kv[0, 0] = 2
    a.kv[1, :P, 0] = v
    ref = v.double().sum(0).cpu().numpy() / (P - 1 + math.exp(gap))
    a.call()
    B.op_sync(stream())
    err = np.abs(a.out.double().cpu().numpy() - ref) / ref
    assert err.max() <= 2.0 ** -35 * math.exp(gap) + 2 * 2.0 ** -11 + 2.0 ** -8 + 2.0 ** -18, err.max()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("state", ["none", "own"])
def test_linattn_nan_decay(B, state, dtype):
    """A NaN decay is not taken for none: its head's outputs and states are NaN, the other heads' keep their bits."""
    lens = [1, 300, 0, 129]
    for step in (False, True):
        a, b = (Lin(B, 3, 64, 128, [1] * 4 if step else lens, dtype, state, log_decay=[-0.1, x, -0.2])
                for x in (float("nan"), -0.3))
        for x in (a, b):
            x.step() if step else x.call()
        B.op_sync(stream())
        assert torch.isnan(a.out[:, 1]).all()
        full = [i for i, n in enumerate(a.lens) if n]
        assert torch.isnan(a.S_out[full, 1]).all()
        assert torch.equal(a.out[:, ::2], b.out[:, ::2]) and torch.equal(a.S_out[:, ::2], b.S_out[:, ::2])
        for i, n in enumerate(a.lens):       # (an empty sequence's state is its initial one)
            if n == 0:
                assert torch.equal(a.S_out[i], a.S_in[i] if a.S_in is not None else torch.zeros_like(a.S_out[i]))


@pytest.mark.parametrize("log_decay", [[-0.7, -0.005], [-3.0, -0.1], [0.0, -0.0004]])
@pytest.mark.parametrize("state", ["none", "own"])
@pytest.mark.parametrize("D", [64, 128])
def test_linattn_f16_sparse_large_elements(B, D, state, log_decay):
    """Two elements in a thousand of q, k and v are 3000 times the others. Outputs keep compare()'s tolerance,
    elements that hold none of the large ones, or whose decay has forgotten them, too. States: a decayed value
    is off by at most 2^-37 of its chunk's largest besides (below |v|'s largest), so the state by that times the
    sum of |k|, decayed from the chunk's end on."""
    a = Lin(B, 2, D, D, [300, 141], "f16", state, log_decay=log_decay, seed=21)
    g = np.random.default_rng(8)
    large = torch.from_numpy(g.random(tuple(a.x.shape)) < 0.002).cuda()
    a.x.copy_(torch.where(large, a.x * 3000, a.x).clamp(-60000, 60000))
    a.scale = 2.0 ** -13
    a.call()
    B.op_sync(stream())
    out, mag, S, A = a.ref()
    got = a.out.double().cpu().numpy()
    tol = 3 * U["f16"] * mag + 1e-6 * mag + 1e-7
    over = np.abs(out) - tol > 65520         # (past f16's largest number)
    assert (got[over] == np.copysign(np.inf, out[over])).all()
    fits = np.abs(out) + tol < 65520
    err = np.abs(got[fits] - out[fits])
    assert fits.mean() > 0.9 and (err <= tol[fits]).all(), (err / (mag[fits] + 1e-30)).max() / U["f16"]
    k, v = (np.abs(t.double().cpu().numpy().reshape(a.R, 2, D)) for t in a.parts()[1:])
    lam = np.exp(a.ld.double().cpu().numpy())
    for s, (r0, n) in enumerate(zip(a.row0, a.lens)):
        floor = np.zeros((2, D))
        for c in range(0, n, 128):
            rows = slice(r0 + c, r0 + min(n, c + 128))
            floor += v[rows].max() * k[rows].sum(0) * (lam ** (n - min(n, c + 128)))[:, None]
        es = np.abs(a.S_out[s].double().cpu().numpy() - S[s])
        assert (es <= (2.0 ** -16 + 2.0 ** -18) * A[s] + 2.0 ** -37 * floor[:, None, :] + 1e-9).all()


@pytest.mark.parametrize("fmt", ["f16", "e4m3"])
@pytest.mark.parametrize("e", [-24, -6, -2, -1, 0, 1, 3, 5])
def test_attention_scores_far_from_zero(B, fmt, e):
    """Equal scores of 2^22 2^e (up to 2^27, where fp32's steps are 8 and more): every weight is the same, whatever
    its rounding, so the result is the values' mean (tol()); and one key behind them that scores a step of its
    type higher (2^12 2^e and more, so it takes all the weight) gives its value, rounded."""
    hd, P = 64, 700
    for one in (False, True):
        if one and e < -2:
            continue
        a = Attn(B, 4, 1, hd, P, [3], fmt, own=False)
        k = torch.full((P, hd), 256.0, dtype=torch.float16)
        if one:
            k[555] += 0.25 if fmt == "f16" else 32
        if fmt == "f16":
            a.kv[0, :P, 0] = k.cuda()
        else:
            k, v = k.cuda(), torch.from_numpy(np.random.default_rng(6).standard_normal((P, hd))).half().cuda()
            B.op_kv_quant_async(k.data_ptr(), v.data_ptr(), B.S1_F16, hd, hd, P, 1, hd, a.kv.data_ptr(),
                                a.scales.data_ptr(), a.cap, 0, stream())
            a.used = (E4M3[a.kv[:, :P].cpu().numpy()] *
                      a.scales[:, :, :P].double().cpu().numpy().transpose(0, 2, 1)[..., None])
        a.x[:] = 256
        a.scale = 2.0 ** e
        a.call()
        B.op_sync(stream())
        got = a.out.double().cpu().numpy()
        ref = a.used[1][555, 0] if one else a.used[1][:, 0].mean(0)
        assert np.abs(got - ref).max() <= a.tol(), (one, np.abs(got - ref).max())
