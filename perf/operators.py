"""Workloads of the operators that serve a batch of questions over one long prefix.

Three families, each with its plain form (elementary torch operations in 32 bits) and the
framework's own calls:

- the 8-bit K/V snapshot: quantising rows as they are written (`kv_write`) and reading them back
  (`kv_read`); e4m3 codes with one power-of-two scale per plane, row and head;
- attention of a batch of sequences that continue one prefix (`attn`): single tokens or question
  suffixes over an f16 or an 8-bit snapshot;
- linear attention with a decay for each head: prompts (`linattn`) and single tokens (`step`).
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
WIDTH = {"f32": 4, "f16": 2, "bf16": 2}


# ---- cases -----------------------------------------------------------------------------------
def listed():
    return [
        # the 27B-class model's prefix of 1536 rows, one attention layer, written into its snapshot
        dict(name="kv_write_27b_prefix", op="kv_write", rows=1536, heads=8, hd=128, dtype="f16", fused=True, pos0=0),
        # a very long context appended behind a short one, rows straight from an fp32 projection
        dict(name="kv_write_long_f32", op="kv_write", rows=100003, heads=4, hd=128, dtype="f32", fused=True, pos0=77),
        # the 4B model's 1024-row prefix read back as f16
        dict(name="kv_read_4b_prefix", op="kv_read", rows=1024, heads=4, hd=128, dtype="f16", fused=False, pos0=0),
        # a long context of 64-wide heads read back for a bf16 consumer
        dict(name="kv_read_long_bf16", op="kv_read", rows=150001, heads=8, hd=64, dtype="bf16", fused=False, pos0=5),
        # the 4B request: three questions of 48 rows over 1024 cached rows (latency counts)
        dict(name="attn_4b_questions", op="attn", fmt="f16", P=1024, lens="48,48,48", gap=0, hq=16, hkv=4, hd=128),
        # the 4B multimodal request: 32 questions of 40 rows over 1280 cached rows
        dict(name="attn_4b_multimodal", op="attn", fmt="f16", P=1280, lens=",".join(["40"] * 32), gap=0, hq=16, hkv=4,
             hd=128),
        # single tokens of 37 sequences over one long 8-bit prefix, the 27B-class heads
        dict(name="attn_tokens_27b_e4m3", op="attn", fmt="e4m3", P=40961, lens=",".join(["1"] * 37), gap=0, hq=40,
             hkv=8, hd=128),
        # ragged questions over a book-length f16 prefix
        dict(name="attn_ragged_long", op="attn", fmt="f16", P=65536,
             lens="120,1,64,33,97,5,40,111,72,18,64,50,88,3,127,129,60,24,9,77,64,31,100,13", gap=0, hq=16, hkv=4,
             hd=128),
        # the 4B model's 1024-row prefix through one linear layer of 16 heads
        dict(name="linattn_4b_prefix", op="linattn", lens="1024", gap=0, heads=16, dk=128, dv=128, dtype="f16",
             state="none", keep=True),
        # three long ragged prompts, 32 heads, each continuing its own state
        dict(name="linattn_long_ragged", op="linattn", lens="9001,130,7345", gap=0, heads=32, dk=128, dv=128,
             dtype="bf16", state="own", keep=True),
        # three one-token questions that continue one prefix state and leave it as it is
        dict(name="step_questions", op="step", n=3, heads=16, dk=128, dv=128, dtype="f16", state="shared", keep=False),
        # a serving batch: one token for each of 255 sequences, every state advanced
        dict(name="step_batch", op="step", n=255, heads=32, dk=128, dv=128, dtype="bf16", state="own", keep=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["kv_write", "kv_read", "attn", "attn", "linattn", "step"])
    if op in ("kv_write", "kv_read"):
        heads, hd = rng.choice([1, 2, 4, 5, 8]), rng.choice([64, 128])
        dtype = rng.choice(["f16", "bf16", "f32"])
        top = min(150000, 480_000_000 // (2 * heads * hd * (1 + WIDTH[dtype])))
        return dict(op=op, rows=_log_int(rng, 1, top), heads=heads, hd=hd, dtype=dtype,
                    fused=rng.random() < 0.5, pos0=rng.choice([0, 0, rng.randint(1, 999)]))
    if op == "attn":
        hq, hkv = rng.choice([(16, 4), (40, 8), (8, 2), (4, 4), (4, 1), (6, 2)])
        hd = rng.choice([64, 128])
        rows = _log_int(rng, 1, 1400)
        if rng.random() < 0.4:
            lens = [1] * min(rows, 256)
        else:
            n = _log_int(rng, 1, min(rows, 48))
            cuts = sorted(rng.randint(0, rows) for _ in range(n - 1))
            lens = [b - a for a, b in zip([0] + cuts, cuts + [rows])]
        total = max(1, sum(lens))
        top = min(65536, int(65536 * 1400 * 16 // (total * hq)), int(80_000_000 // (hkv * hd)))
        return dict(op=op, fmt=rng.choice(["f16", "e4m3"]), P=_log_int(rng, 1, max(16, top)),
                    lens=",".join(map(str, lens)), gap=rng.choice([0, 0, rng.randint(1, 9)]), hq=hq, hkv=hkv, hd=hd)
    heads, dk, dv = rng.choice([1, 4, 8, 16, 32]), rng.choice([64, 128]), rng.choice([64, 128])
    dtype, state = rng.choice(["f16", "bf16"]), rng.choice(["none", "own", "shared"])
    if op == "linattn":
        rows = _log_int(rng, 1, 16000)
        n = _log_int(rng, 1, min(rows, 24))
        cuts = sorted(rng.randint(0, rows) for _ in range(n - 1))
        lens = [b - a for a, b in zip([0] + cuts, cuts + [rows])]
        return dict(op=op, lens=",".join(map(str, lens)), gap=rng.choice([0, 0, rng.randint(1, 9)]), heads=heads,
                    dk=dk, dv=dv, dtype=dtype, state=state, keep=rng.random() < 0.8)
    return dict(op=op, n=_log_int(rng, 1, 250), heads=heads, dk=dk, dv=dv, dtype=dtype, state=state,
                keep=rng.random() < 0.7)


def _lens(case):
    """Row counts and first rows of the packed sequences (`gap` unused rows between them)."""
    lens = [int(x) for x in case["lens"].split(",")]
    row0, at = [], 0
    for n in lens:
        row0.append(at)
        at += n + case["gap"]
    return lens, row0, max(1, at)


# ---- inputs ----------------------------------------------------------------------------------
def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _quantise(x):
    """[.., hd] fp32 -> e4m3 codes and one power-of-two scale per vector."""
    a = x.abs()
    a = torch.where(torch.isfinite(a), a, torch.zeros_like(a)).amax(-1)
    m, e = torch.frexp(a)                         # a = m 2^e, 1/2 <= m < 1; 448 = 0.875 * 2^9
    E = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-126)
    E = torch.where(a > 0, E, torch.zeros_like(E))
    y = torch.ldexp(x, -E[..., None]).clamp(-448.0, 448.0)
    return y.to(torch.float8_e4m3fn), torch.ldexp(torch.ones_like(a), E)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, s = case["op"], dict(case)
    if op in ("kv_write", "kv_read"):
        n, H, hd, dt = case["rows"], case["heads"], case["hd"], DTYPES[case["dtype"]]
        cap = case["pos0"] + n + 64
        s["cap"] = cap
        if op == "kv_write":
            # post-rotation keys and values: unit scale, a few channels with large values
            boost = torch.ones(H * hd, device="cuda")
            boost[torch.randint(0, H * hd, (max(1, H * hd // 64),), generator=g, device="cuda")] = 20.0
            if case["fused"]:      # k and v as slices of one projection's rows
                x = (_randn(g, n, 2 * H * hd) * torch.cat([boost, torch.ones_like(boost)])).to(dt)
                s["k"], s["v"] = x[:, :H * hd], x[:, H * hd:]
            else:
                s["k"], s["v"] = (_randn(g, n, H * hd) * boost).to(dt), _randn(g, n, H * hd, dtype=dt)
            s["codes"] = torch.zeros(2, cap, H, hd, device="cuda", dtype=torch.uint8)
            s["scales"] = torch.zeros(2, H, cap, device="cuda")
        else:
            c, sc = _quantise(_randn(g, 2, cap, H, hd))
            s["codes"], s["scales"] = c.view(torch.uint8), sc.transpose(1, 2).contiguous()
            s["k"], s["v"] = (torch.zeros(n, H * hd, device="cuda", dtype=dt) for _ in range(2))
    elif op == "attn":
        lens, row0, R = _lens(case)
        hq, hkv, hd, P = case["hq"], case["hkv"], case["hd"], case["P"]
        cap = P + 17
        # q, k, v as slices of one projection's rows; the first prefix rows draw extra attention
        x = _randn(g, R, (hq + 2 * hkv) * hd, dtype=torch.float16)
        s["q"], s["kn"], s["vn"] = x[:, :hq * hd], x[:, hq * hd:(hq + hkv) * hd], x[:, (hq + hkv) * hd:]
        kv = _randn(g, 2, cap, hkv, hd)
        kv[0, :4] *= 1.5
        if case["fmt"] == "f16":
            s["kv"], s["scales"] = kv.half(), None
        else:
            c, sc = _quantise(kv)
            s["kv"], s["scales"] = c.view(torch.uint8), sc.transpose(1, 2).contiguous()
        del kv
        s["cap"], s["out"] = cap, torch.zeros(R, hq, hd, device="cuda", dtype=torch.float16)
    else:
        H, dk, dv, dt = case["heads"], case["dk"], case["dv"], DTYPES[case["dtype"]]
        if op == "linattn":
            lens, _, R = _lens(case)
            n = len(lens)
        else:
            n = R = case["n"]
        x = _randn(g, R, H * (2 * dk + dv), dtype=dt)
        s["q"], s["k"], s["v"] = x[:, :H * dk], x[:, H * dk:2 * H * dk], x[:, 2 * H * dk:]
        # geometric slopes over the heads, from a memory of one token to one of hundreds
        h = torch.arange(1, H + 1, device="cuda", dtype=torch.float32)
        s["log_decay"] = -torch.exp2(-8.0 * h / H)
        shape = {"none": None, "shared": (1, H, dv, dk), "own": (n, H, dv, dk)}[case["state"]]
        s["s_in"] = None if shape is None else _randn(g, *shape) * 3.0
        s["s_out"] = torch.zeros(n, H, dv, dk, device="cuda") if case["keep"] else None
        s["out"] = torch.zeros(R, H, dv, device="cuda", dtype=dt)
    if own:
        _prepare_own(case, s)
    return s


# ---- the framework's calls -------------------------------------------------------------------
def _prepare_own(case, s):
    import numpy as np
    from prefill_only_decision_gb300 import binding as B
    s["B"] = B
    s["dt"] = {"f32": B.S1_F32, "f16": B.S1_F16, "bf16": B.S1_BF16}.get(case.get("dtype"))
    if "lens" in case:
        lens, row0, _ = _lens(case)
        s["n_rows"] = np.asarray(lens, np.int32)
        s["row0"] = np.asarray(row0, np.int32)
    if case["op"] == "attn":
        nb = B.op_attention_shared_workspace(s["n_rows"], case["P"], case["hq"], case["hkv"], case["hd"])
        s["ws"] = torch.empty(max(16, nb), device="cuda", dtype=torch.uint8)
    elif case["op"] == "linattn":
        nb = B.op_linattn_workspace(s["n_rows"], case["heads"], case["dk"], case["dv"])
        s["ws"] = torch.empty(max(16, nb), device="cuda", dtype=torch.uint8)


def _run_own(s):
    B, op = s["B"], s["op"]
    stream = torch.cuda.current_stream().cuda_stream
    if op == "kv_write":
        B.op_kv_quant_async(s["k"].data_ptr(), s["v"].data_ptr(), s["dt"], s["k"].stride(0), s["v"].stride(0),
                            s["rows"], s["heads"], s["hd"], s["codes"].data_ptr(), s["scales"].data_ptr(), s["cap"],
                            s["pos0"], stream)
        return s["codes"].view(torch.float8_e4m3fn), s["scales"]
    if op == "kv_read":
        B.op_kv_dequant_async(s["codes"].data_ptr(), s["scales"].data_ptr(), s["cap"], s["pos0"], s["rows"],
                              s["heads"], s["hd"], s["k"].data_ptr(), s["v"].data_ptr(), s["dt"], s["k"].stride(0),
                              s["v"].stride(0), stream)
        return s["k"], s["v"]
    if op == "attn":
        B.op_attention_shared_async(s["q"].data_ptr(), s["q"].stride(0), s["kn"].data_ptr(), s["vn"].data_ptr(),
                                    s["kn"].stride(0), s["row0"], s["n_rows"], s["kv"].data_ptr(),
                                    0 if s["scales"] is None else s["scales"].data_ptr(),
                                    B.S1_KV_F16 if s["scales"] is None else B.S1_KV_E4M3, s["P"], s["cap"], s["hq"],
                                    s["hkv"], s["hd"], s["hd"] ** -0.5, s["out"].data_ptr(), s["ws"].data_ptr(),
                                    s["ws"].numel(), stream)
        return s["out"]
    H, dk, dv = s["heads"], s["dk"], s["dv"]
    s_in = 0 if s["s_in"] is None else s["s_in"].data_ptr()
    s_in_stride = H * dv * dk if s["state"] == "own" else 0
    s_out = 0 if s["s_out"] is None else s["s_out"].data_ptr()
    if op == "linattn":
        B.op_linattn_async(s["q"].data_ptr(), s["k"].data_ptr(), s["v"].data_ptr(), s["dt"], s["q"].stride(0),
                           s["k"].stride(0), s["v"].stride(0), s["log_decay"].data_ptr(), s["row0"], s["n_rows"], H,
                           dk, dv, dk ** -0.5, s_in, s_in_stride, s_out, s["out"].data_ptr(), s["ws"].data_ptr(),
                           s["ws"].numel(), stream)
    else:
        B.op_linattn_step_async(s["q"].data_ptr(), s["k"].data_ptr(), s["v"].data_ptr(), s["dt"], s["q"].stride(0),
                                s["k"].stride(0), s["v"].stride(0), s["log_decay"].data_ptr(), s["n"], H, dk, dv,
                                dk ** -0.5, s_in, s_in_stride, s_out, s["out"].data_ptr(), stream)
    return s["out"] if s["s_out"] is None else (s["out"], s["s_out"])


# ---- plain forms -----------------------------------------------------------------------------
def run(state):
    if own:
        return _run_own(state)
    s, op = state, state["op"]
    if op == "kv_write":
        n, H, hd, p = s["rows"], s["heads"], s["hd"], s["pos0"]
        for plane, x in enumerate((s["k"], s["v"])):
            c, sc = _quantise(x.float().view(n, H, hd))
            s["codes"][plane, p:p + n] = c.view(torch.uint8)
            s["scales"][plane, :, p:p + n] = sc.t()
        return s["codes"].view(torch.float8_e4m3fn), s["scales"]
    if op == "kv_read":
        n, H, hd, p = s["rows"], s["heads"], s["hd"], s["pos0"]
        top = torch.finfo(s["k"].dtype).max
        for plane, y in enumerate((s["k"], s["v"])):
            c = s["codes"][plane, p:p + n].view(torch.float8_e4m3fn).float()
            x = c * s["scales"][plane, :, p:p + n].t()[:, :, None]
            y.copy_(x.clamp(-top, top).view(n, H * hd))
        return s["k"], s["v"]
    if op == "attn":
        return _plain_attn(s)
    return _plain_linattn(s) if op == "linattn" else _plain_step(s)


def _plain_attn(s):
    lens, row0, _ = _lens(s)
    hq, hkv, hd, P = s["hq"], s["hkv"], s["hd"], s["P"]
    G, scale = hq // hkv, s["hd"] ** -0.5
    dev = s["q"].device
    rows = torch.cat([torch.arange(a, a + n, device=dev) for a, n in zip(row0, lens)])
    seq = torch.repeat_interleave(torch.arange(len(lens), device=dev), torch.tensor(lens, device=dev))
    N = rows.numel()
    if N == 0:
        return s["out"]
    seen = (seq[:, None] == seq[None, :]) & (rows[:, None] >= rows[None, :])
    seen = seen[:, None, :].expand(N, G, N).reshape(N * G, N)
    q = s["q"].float().view(-1, hq, hd)[rows]
    kn, vn = s["kn"].float().view(-1, hkv, hd)[rows], s["vn"].float().view(-1, hkv, hd)[rows]
    for h in range(hkv):
        kp, vp = s["kv"][0, :P, h], s["kv"][1, :P, h]
        if s["scales"] is not None:
            kp, vp = ((c.view(torch.float8_e4m3fn).float() * s["scales"][i, h, :P, None]).half()
                      for i, c in enumerate((kp, vp)))
        qh = q[:, h * G:(h + 1) * G].reshape(N * G, hd) * scale
        a = torch.cat([qh @ kp.float().t(), (qh @ kn[:, h].t()).masked_fill(~seen, -math.inf)], 1)
        a = torch.exp(a - a.amax(1, keepdim=True))
        o = (a[:, :P] @ vp.float() + a[:, P:] @ vn[:, h]) / a.sum(1, keepdim=True)
        s["out"][rows, h * G:(h + 1) * G] = o.view(N, G, hd).half()
    return s["out"]


def _first_state(s, i):
    H, dk, dv = s["heads"], s["dk"], s["dv"]
    if s["s_in"] is None:
        return torch.zeros(H, dv, dk, device=s["q"].device)
    return s["s_in"][i if s["state"] == "own" else 0]


def _plain_linattn(s):
    """Chunks of 128 rows: within a chunk the masked products, between chunks the state."""
    lens, row0, _ = _lens(s)
    H, dk, dv, C = s["heads"], s["dk"], s["dv"], 128
    q = s["q"].float().view(-1, H, dk) * dk ** -0.5
    k, v = s["k"].float().view(-1, H, dk), s["v"].float().view(-1, H, dv)
    t = torch.arange(C, device=q.device, dtype=torch.float32)
    w = s["log_decay"][:, None] * (t[None, :] + 1)                       # log lam^(i+1)       [H, C]
    lag = t[:, None] - t[None, :]
    D = torch.exp(s["log_decay"][:, None, None] * lag.clamp(min=0)) * (lag >= 0)
    for i, (a, n) in enumerate(zip(row0, lens)):
        S = _first_state(s, i).clone()
        for c in range(0, n, C):
            m = min(C, n - c)
            Q, K, V = (x[a + c:a + c + m].transpose(0, 1) for x in (q, k, v))
            o = torch.exp(w[:, :m, None]) * (Q @ S.transpose(1, 2)) + ((Q @ K.transpose(1, 2)) * D[:, :m, :m]) @ V
            back = torch.exp(s["log_decay"][:, None] * (m - 1 - t[None, :m]))
            S = torch.exp(w[:, m - 1, None, None]) * S + (V * back[..., None]).transpose(1, 2) @ K
            s["out"][a + c:a + c + m] = o.transpose(0, 1).to(s["out"].dtype)
        if s["s_out"] is not None:
            s["s_out"][i] = S
    return s["out"] if s["s_out"] is None else (s["out"], s["s_out"])


def _plain_step(s):
    n, H, dk, dv = s["n"], s["heads"], s["dk"], s["dv"]
    q = s["q"].float().view(n, H, 1, dk) * dk ** -0.5
    k, v = s["k"].float().view(n, H, 1, dk), s["v"].float().view(n, H, dv, 1)
    S = v * k
    if s["s_in"] is not None:
        S = S + torch.exp(s["log_decay"])[:, None, None] * s["s_in"]
    s["out"].copy_((S * q).sum(-1))
    if s["s_out"] is None:
        return s["out"]
    s["s_out"].copy_(S)
    return s["out"], s["s_out"]


# ---- necessary work --------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op in ("kv_write", "kv_read"):
        n = 2 * case["rows"] * case["heads"]
        return {"bytes": n * case["hd"] * (1 + WIDTH[case["dtype"]]) + 4 * n, "flops": 2 * n * case["hd"]}
    if op == "attn":
        lens, hq, hkv, hd = _lens(case)[0], case["hq"], case["hkv"], case["hd"]
        R = sum(lens)
        prefix = 2 * case["P"] * hkv * (2 * hd if case["fmt"] == "f16" else hd + 4)
        keys = sum(n * case["P"] + n * (n + 1) // 2 for n in lens)
        return {"bytes": prefix + 2 * R * hd * (2 * hq + 2 * hkv), "flops": 4 * hd * hq * keys}
    H, dk, dv, wd = case["heads"], case["dk"], case["dv"], WIDTH[case["dtype"]]
    if op == "linattn":
        lens = _lens(case)[0]
        R, n = sum(lens), len(lens)
    else:
        R = n = case["n"]
    states = {"none": 0, "shared": 1, "own": n}[case["state"]] + (n if case["keep"] else 0)
    return {"bytes": R * H * wd * (2 * dk + 2 * dv) + 4 * states * H * dk * dv + 4 * H, "flops": 4 * R * H * dk * dv}


# ---- the definitions in 64 bits --------------------------------------------------------------
def _grid(x, bits, lowest, top):
    """Round to `bits` significant bits (ties to even) with exponents from `lowest`, at most `top`."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -1000))).clamp(min=lowest)
    step = torch.exp2(e - (bits - 1))
    return (torch.round(x / step) * step).clamp(-top, top)


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    d = torch.float64
    if op == "kv_write":
        n, H, hd, p, cap = case["rows"], case["heads"], case["hd"], case["pos0"], s["cap"]
        values = torch.zeros(2, cap, H, hd, device="cuda", dtype=d)
        scales = torch.zeros(2, H, cap, device="cuda", dtype=d)
        for plane in range(2):
            x = s["kv"[plane]].to(d).reshape(n, H, hd)
            a = x.abs().amax(2)
            sc = torch.exp2(torch.floor(torch.log2(a / 448.0)) - 1)      # at or below the wanted power of two
            for _ in range(3):
                sc = torch.where(448.0 * sc < a, 2 * sc, sc)
            values[plane, p:p + n] = _grid(x / sc[..., None], 4, -6, 448.0)
            scales[plane, :, p:p + n] = sc.t()
        return values, scales
    if op == "kv_read":
        n, H, hd, p = case["rows"], case["heads"], case["hd"], case["pos0"]
        b = s["codes"][:, p:p + n].to(torch.int32)
        sign, e, m = b >> 7, (b >> 3) & 15, b & 7
        x = torch.where(e > 0, (8 + m).to(d) * torch.exp2(e.to(d) - 10), m.to(d) * 2.0 ** -9) * (1 - 2 * sign)
        x = x * s["scales"][:, :, p:p + n].to(d).permute(0, 2, 1)[..., None]
        return x[0].reshape(n, H * hd), x[1].reshape(n, H * hd)
    if op == "attn":
        lens, row0, R = _lens(case)
        hq, hkv, hd, P = case["hq"], case["hkv"], case["hd"], case["P"]
        out = torch.zeros(R, hq, hd, device="cuda", dtype=d)
        for h in range(hkv):
            k, v = s["kv"][0, :P, h], s["kv"][1, :P, h]
            if s["scales"] is not None:
                k = k.view(torch.float8_e4m3fn).to(d) * s["scales"][0, h, :P, None].to(d)
                v = v.view(torch.float8_e4m3fn).to(d) * s["scales"][1, h, :P, None].to(d)
            k, v = k.to(d), v.to(d)
            for a, n in zip(row0, lens):
                if n == 0:
                    continue
                ko, vo = (x[a:a + n, h * hd:(h + 1) * hd].to(d) for x in (s["kn"], s["vn"]))
                future = torch.ones(n, n, device="cuda", dtype=torch.bool).triu(1)
                for j in range(h * hq // hkv, (h + 1) * hq // hkv):
                    qj = s["q"][a:a + n, j * hd:(j + 1) * hd].to(d) / math.sqrt(hd)
                    z = torch.cat([qj @ k.t(), (qj @ ko.t()).masked_fill(future, -math.inf)], 1)
                    w = torch.softmax(z, 1)
                    out[a:a + n, j] = w[:, :P] @ v + w[:, P:] @ vo
        return out
    H, dk, dv = case["heads"], case["dk"], case["dv"]
    if op == "linattn":
        lens, row0, R = _lens(case)
    else:
        R = case["n"]
        lens, row0 = [1] * R, list(range(R))
    lam = torch.exp(s["log_decay"].to(d))[:, None, None]
    q, k, v = (s[x].to(d).reshape(R, H, -1) for x in "qkv")
    q = q / math.sqrt(dk)
    out = torch.zeros(R, H, dv, device="cuda", dtype=d)
    last = torch.zeros(len(lens), H, dv, dk, device="cuda", dtype=d)
    for i, (a, n) in enumerate(zip(row0, lens)):
        S = last[i]
        if s["s_in"] is not None:
            S.copy_(s["s_in"][i if case["state"] == "own" else 0])
        for t in range(a, a + n):        # one token after the other, as the operator is defined
            S.mul_(lam).add_(v[t][:, :, None] * k[t][:, None, :])
            out[t] = torch.matmul(S, q[t][:, :, None])[..., 0]
    return (out, last) if case["keep"] else out
