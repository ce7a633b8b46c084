"""Workloads of the operators around a paged K/V cache.

Four families, each with its plain form (elementary torch operations) and the framework's own calls:

- rotary positions with one or several axes (`rope`);
- keys and values appended to a paged cache, rotated on the way, with the rotated queries (`append`);
- attention of one new token of each sequence over its pages (`step`);
- attention of prompt rows over their pages, with a sliding window and a few first rows that stay
  visible, or without (`prompt`).

A cache holds `[2, n_pages, Hkv, page_rows, hd]` elements (K plane, V plane) and a table of page ids
for each sequence; an 8-bit cache has e4m3 codes and a power-of-two scale for each row and head.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
WIDTH = {"f32": 4, "f16": 2, "bf16": 2, "e4m3": 1}
THETA = 1.0e6


# ---- cases -----------------------------------------------------------------------------------
def listed():
    return [
        # the 4B multimodal request's rows (1024 image patches, 256 tokens): q and k heads of the fused projection
        dict(name="rope_4b_multimodal", op="rope", rows=1280, heads=20, hd=128, rot=128, axes=3, mix=False, src="f16",
             dst="f16"),
        # a long video: fp32 projection rows, half of each head rotated, the three axes taking turns over the pairs
        dict(name="rope_video_long", op="rope", rows=50001, heads=48, hd=128, rot=64, axes=3, mix=True, src="f32",
             dst="bf16"),
        # one token for each of 37 sequences, the 27B-class heads (latency counts)
        dict(name="append_tokens_27b", op="append", seqs=37, rows=37, top=40000, hq=40, hkv=8, hd=128, rot=128, axes=1,
             src="f16", fmt="f16", page=16),
        # ragged multimodal prompts straight from an fp32 projection
        dict(name="append_prompts_f32", op="append", seqs=9, rows=12345, top=3000, hq=16, hkv=4, hd=128, rot=128,
             axes=3, src="f32", fmt="bf16", page=64),
        # book-length prompts into an 8-bit cache
        dict(name="append_long_e4m3", op="append", seqs=5, rows=70001, top=1000, hq=16, hkv=4, hd=128, rot=128, axes=1,
             src="f16", fmt="e4m3", page=32),
        # three one-token questions over about the 4B model's 1024-row prefix, a cache of their own each
        dict(name="step_4b_questions", op="step", seqs=3, low=1000, top=1100, hq=16, hkv=4, hd=128, fmt="f16", page=16,
             window=0, sinks=0),
        # a serving batch over ragged long contexts, the 27B-class heads
        dict(name="step_ragged_27b", op="step", seqs=61, low=1, top=32768, hq=40, hkv=8, hd=128, fmt="bf16", page=64,
             window=0, sinks=0),
        # one token over a very long 8-bit cache
        dict(name="step_one_long_e4m3", op="step", seqs=1, low=200001, top=200001, hq=16, hkv=4, hd=128, fmt="e4m3",
             page=128, window=0, sinks=0),
        # a large batch that sees its last 1024 rows and the first 4
        dict(name="step_window_batch", op="step", seqs=255, low=1, top=20000, hq=16, hkv=4, hd=64, fmt="f16", page=16,
             window=1024, sinks=4),
        # the 4B model's 1024-row prefix under a short window
        dict(name="prompt_4b_prefix_window", op="prompt", lens="1024", pos0="0", gap=0, hq=16, hkv=4, hd=128, fmt="f16",
             page=16, window=256, sinks=4),
        # long ragged prompts, two of them continued, under a window
        dict(name="prompt_window_long", op="prompt", lens="9001,130,7345", pos0="0,5000,12001", gap=3, hq=16, hkv=4,
             hd=128, fmt="bf16", page=64, window=2048, sinks=16),
        # a chunk of a prompt that continues a very long one and sees all of it
        dict(name="prompt_chunk_27b", op="prompt", lens="512", pos0="50000", gap=0, hq=40, hkv=8, hd=128, fmt="f16",
             page=32, window=0, sinks=0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


HEADS = [(16, 4), (40, 8), (8, 2), (4, 4), (6, 2), (16, 1), (12, 3)]


def draw(rng):
    op = rng.choice(["rope", "append", "step", "step", "prompt", "prompt"])
    hd = rng.choice([64, 128])
    page = rng.choice([16, 32, 64, 128])
    if op == "rope":
        heads, axes = rng.choice([1, 3, 10, 20, 48]), rng.choice([1, 2, 3, 4])
        src = rng.choice(["f16", "bf16", "f32"])
        top = min(100_000, 300_000_000 // (heads * hd))
        return dict(op=op, rows=_log_int(rng, 1, top), heads=heads, hd=hd, rot=rng.choice([hd, hd, hd // 2, hd // 4]),
                    axes=axes, mix=rng.random() < 0.5, src=src, dst=rng.choice(["f16", "bf16"]) if src == "f32" else src)
    hq, hkv = rng.choice(HEADS)
    if op == "append":
        top = min(70_000, 215_000_000 // ((hq + 2 * hkv) * hd))
        rows = _log_int(rng, 1, top)
        seqs = rows if rng.random() < 0.3 and rows <= 300 else _log_int(rng, 1, min(rows, 40))
        return dict(op=op, seqs=seqs, rows=rows, top=rng.choice([0, 100, 3001]), hq=hq, hkv=hkv, hd=hd,
                    rot=rng.choice([hd, hd, hd // 2]), axes=rng.choice([1, 1, 3]), src=rng.choice(["f16", "bf16", "f32"]),
                    fmt=rng.choice(["f16", "bf16", "e4m3"]), page=page)
    fmt = rng.choice(["f16", "bf16", "e4m3"]) if op == "step" else rng.choice(["f16", "bf16"])
    window = rng.choice([0, 0, _log_int(rng, 1, 5000)])
    sinks = rng.choice([0, 4, rng.randint(1, 200)]) if window else 0
    if op == "step":
        seqs = _log_int(rng, 1, 300)
        top = min(200_000, 2_000_000_000 // (seqs * hkv * hd * 2))
        return dict(op=op, seqs=seqs, low=1, top=_log_int(rng, 1, top), hq=hq, hkv=hkv, hd=hd, fmt=fmt, page=page,
                    window=window, sinks=sinks)
    rows = _log_int(rng, 1, 12000)
    n = _log_int(rng, 1, min(rows, 20))
    cuts = sorted(rng.randint(0, rows) for _ in range(n - 1))
    lens = [b - a for a, b in zip([0] + cuts, cuts + [rows])]
    # rows x heads x keys at most those of the largest listed case
    top = int(512 * 50000 * 40 // (rows * hq)) - rows // 2
    pos0 = [rng.choice([0, _log_int(rng, 1, max(1, min(60000, top)))]) for _ in lens]
    return dict(op=op, lens=",".join(map(str, lens)), pos0=",".join(map(str, pos0)), gap=rng.choice([0, rng.randint(1, 9)]),
                hq=hq, hkv=hkv, hd=hd, fmt=fmt, page=page, window=window, sinks=sinks)


# ---- what a case's sizes mean ----------------------------------------------------------------
def _append_rows(case):
    """Rows of each sequence and the position at which its rows start."""
    r = random.Random(case["rows"] * 1009 + case["seqs"])
    n, rows = case["seqs"], case["rows"]
    cuts = sorted(r.sample(range(1, rows), n - 1))
    lens = [b - a for a, b in zip([0] + cuts, cuts + [rows])]
    return lens, [r.randint(0, case["top"]) for _ in lens]


def _step_pos(case):
    """The position of each sequence's token: the rows before it are cached, too."""
    r = random.Random(case["seqs"] * 1013 + case["top"])
    return [r.randint(case["low"], case["top"]) - 1 for _ in range(case["seqs"])]


def _prompts(case):
    """Row counts, first rows and first positions of the packed sequences (`gap` unused rows between them)."""
    lens = [int(x) for x in case["lens"].split(",")]
    pos0 = [int(x) for x in case["pos0"].split(",")]
    row0, at = [], 0
    for n in lens:
        row0.append(at)
        at += n + case["gap"]
    return lens, row0, pos0, max(1, at)


def _axis_of(pairs, axes, mix):
    """The position axis of each rotated pair: the axes take turns, or have a run of pairs each."""
    if mix:
        return [i % axes for i in range(pairs)]
    return [min(axes - 1, i * axes // pairs) for i in range(pairs)]


# ---- inputs ----------------------------------------------------------------------------------
def _randn(g, *shape, dtype=torch.float32):
    out = torch.empty(*shape, device="cuda", dtype=dtype)
    flat, step = out.view(-1), 1 << 28
    for i in range(0, flat.numel(), step):
        n = min(step, flat.numel() - i)
        flat[i:i + n] = torch.randn(n, generator=g, device="cuda", dtype=torch.float32)
    return out


def _quantise(x):
    """[.., hd] fp32 -> e4m3 codes and one power-of-two scale per vector."""
    a = x.abs().amax(-1)
    m, e = torch.frexp(a)                         # a = m 2^e, 1/2 <= m < 1; 448 = 0.875 * 2^9
    E = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-126)
    E = torch.where(a > 0, E, torch.zeros_like(E))
    y = torch.ldexp(x, -E[..., None]).clamp(-448.0, 448.0)
    return y.to(torch.float8_e4m3fn), torch.ldexp(torch.ones_like(a), E)


def _positions(g, axes, rows, first):
    """[axes, rows] positions: time runs on, the others move over a grid as patches of a picture do."""
    t = torch.arange(rows, device="cuda", dtype=torch.int32)
    out = [t + first]
    for a in range(1, axes):
        out.append((t // 37 ** (a - 1)) % 37 + torch.randint(0, 1000, (1,), generator=g, device="cuda", dtype=torch.int32))
    return torch.stack(out)


def _tables(g, s, rows_of):
    """Page tables over one pool, pages handed out in no particular order, a few left over."""
    page = s["page"]
    need = [(n + page - 1) // page for n in rows_of]
    s["n_pages"], cols = sum(need) + 3, max(1, max(need))
    ids = torch.randperm(s["n_pages"], generator=g, device="cuda").to(torch.int32)
    s["table"] = torch.full((len(need), cols), -1, device="cuda", dtype=torch.int32)
    at = 0
    for i, n in enumerate(need):
        s["table"][i, :n] = ids[at:at + n]
        at += n


def _filled_cache(g, s):
    """Pages that hold rows already (the rest of a page, too: what was there before)."""
    shape = (2, s["n_pages"], s["hkv"], s["page"], s["hd"])
    if s["fmt"] != "e4m3":
        s["cache"], s["scales"] = _randn(g, *shape, dtype=DTYPES[s["fmt"]]), None
    else:
        s["cache"] = torch.empty(*shape, device="cuda", dtype=torch.uint8)
        s["scales"] = torch.empty(*shape[:-1], device="cuda")
        step = max(1, (1 << 26) // (s["hkv"] * s["page"] * s["hd"]))
        for plane in range(2):
            for p in range(0, s["n_pages"], step):
                c, sc = _quantise(_randn(g, min(step, s["n_pages"] - p), *shape[2:]))
                s["cache"][plane, p:p + step], s["scales"][plane, p:p + step] = c.view(torch.uint8), sc
    first = s["table"][:, 0]
    first = first[first >= 0].long()               # the first rows draw extra attention
    if s["fmt"] != "e4m3":
        s["cache"][0, first, :, :4] *= 1.5
    else:
        s["scales"][0, first, :, :4] *= 2.0


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, s = case["op"], dict(case)
    hd = s["hd"]
    if op in ("rope", "append"):
        pairs = s["rot"] // 2
        s["inv_freq"] = [THETA ** (-i / pairs) for i in range(pairs)]
        s["axis"] = _axis_of(pairs, s["axes"], case.get("mix", False))
        s["axis_t"] = torch.tensor(s["axis"], device="cuda")
        s["freq_t"] = torch.tensor(s["inv_freq"], device="cuda", dtype=torch.float64)
    if op == "rope":
        x = _randn(g, s["rows"], (s["heads"] + 4) * hd, dtype=DTYPES[s["src"]])
        s["x"] = x[:, :s["heads"] * hd]            # the q and k part of a fused projection's rows
        s["pos"] = _positions(g, s["axes"], s["rows"], 100_000)
        s["out"] = torch.zeros(s["rows"], s["heads"] * hd, device="cuda", dtype=DTYPES[s["dst"]])
    elif op == "append":
        lens, first = _append_rows(case)
        hq, hkv = s["hq"], s["hkv"]
        x = _randn(g, s["rows"], (hq + 2 * hkv) * hd, dtype=DTYPES[s["src"]])
        s["q"], s["k"], s["v"] = x[:, :hq * hd], x[:, hq * hd:(hq + hkv) * hd], x[:, (hq + hkv) * hd:]
        _tables(g, s, [a + n for a, n in zip(first, lens)])
        n_rows = torch.tensor(lens, device="cuda")
        s["seq"] = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), n_rows).to(torch.int32)
        s["at"] = torch.cat([torch.arange(a, a + n, device="cuda", dtype=torch.int32) for a, n in zip(first, lens)])
        s["pos"] = s["at"][None] if s["axes"] == 1 else _positions(g, s["axes"], s["rows"], 0)
        shape = (2, s["n_pages"], hkv, s["page"], hd)
        q_dtype = torch.float16 if s["fmt"] == "e4m3" else DTYPES[s["fmt"]]
        s["q_out"] = torch.zeros(s["rows"], hq * hd, device="cuda", dtype=q_dtype)
        s["cache"] = torch.zeros(*shape, device="cuda", dtype=torch.uint8 if s["fmt"] == "e4m3" else q_dtype)
        s["scales"] = torch.zeros(*shape[:-1], device="cuda") if s["fmt"] == "e4m3" else None
    else:
        dt = torch.float16 if s["fmt"] == "e4m3" else DTYPES[s["fmt"]]
        if op == "step":
            pos = _step_pos(case)
            s["pos"] = torch.tensor(pos, device="cuda", dtype=torch.int32)
            R, ends = len(pos), [p + 1 for p in pos]
        else:
            lens, _, pos0, R = _prompts(case)
            ends = [p + n for p, n in zip(pos0, lens)]
        _tables(g, s, ends)
        s["q"] = _randn(g, R, s["hq"] * hd, dtype=dt)
        _filled_cache(g, s)
        s["out"] = torch.zeros(R, s["hq"], hd, device="cuda", dtype=dt)
    if own:
        _prepare_own(case, s)
    return s


# ---- the framework's calls -------------------------------------------------------------------
def _prepare_own(case, s):
    import numpy as np
    from prefill_only_decision_gb300 import binding as B
    s["B"] = B
    code = {"f32": B.S1_F32, "f16": B.S1_F16, "bf16": B.S1_BF16}
    op = s["op"]
    if op in ("rope", "append"):
        s["rope"] = B.Rope(s["inv_freq"], s["axis"])
        s["dt"] = code[s["src"]]
    if op == "rope":
        s["dt_out"] = code[s["dst"]]
        return
    fmt = {"f16": B.S1_KV_F16, "bf16": B.S1_KV_BF16, "e4m3": B.S1_KV_E4M3}[s["fmt"]]
    s["q_dt"] = B.S1_BF16 if s["fmt"] == "bf16" else B.S1_F16
    s["pages"] = B.KvPages(s["cache"].data_ptr(), 0 if s["scales"] is None else s["scales"].data_ptr(), fmt,
                           s["n_pages"], s["page"], s["hkv"], s["hd"], s["table"].data_ptr(), s["table"].shape[0],
                           s["table"].shape[1])
    nb = 0
    if op == "step":
        nb = B.op_attention_paged_step_workspace(s["seqs"], s["hq"], s["hkv"], s["hd"])
    elif op == "prompt":
        lens, row0, pos0, _ = _prompts(case)
        s["n_rows"], s["row0"], s["pos0_h"] = (np.asarray(x, np.int32) for x in (lens, row0, pos0))
        nb = B.op_attention_paged_workspace(s["n_rows"], s["pos0_h"], s["hq"], s["hkv"], s["hd"], s["window"], s["sinks"])
    s["ws"] = torch.empty(max(16, nb), device="cuda", dtype=torch.uint8)


def _run_own(s):
    B, op = s["B"], s["op"]
    stream = torch.cuda.current_stream().cuda_stream
    if op == "rope":
        B.op_rope_async(s["x"].data_ptr(), s["dt"], s["x"].stride(0), s["rows"], s["heads"], s["hd"], s["rope"],
                        s["pos"].data_ptr(), s["pos"].stride(0), s["out"].data_ptr(), s["dt_out"], s["out"].stride(0),
                        stream)
        return s["out"]
    if op == "append":
        B.op_kv_append_async(s["q"].data_ptr(), s["k"].data_ptr(), s["v"].data_ptr(), s["dt"], s["q"].stride(0),
                             s["k"].stride(0), s["v"].stride(0), s["rows"], s["hq"], s["rope"], s["pos"].data_ptr(),
                             s["pos"].stride(0), s["seq"].data_ptr(), s["at"].data_ptr(), s["pages"],
                             s["q_out"].data_ptr(), s["q_dt"], stream)
        return _append_out(s)
    if op == "step":
        B.op_attention_paged_step_async(s["q"].data_ptr(), s["q_dt"], s["q"].stride(0), s["seqs"], s["hq"], s["pages"],
                                        s["pos"].data_ptr(), s["window"], s["sinks"], s["hd"] ** -0.5,
                                        s["out"].data_ptr(), s["ws"].data_ptr(), s["ws"].numel(), stream)
    else:
        B.op_attention_paged_async(s["q"].data_ptr(), s["q_dt"], s["q"].stride(0), s["row0"], s["n_rows"], s["pos0_h"],
                                   s["hq"], s["pages"], s["window"], s["sinks"], s["hd"] ** -0.5, s["out"].data_ptr(),
                                   s["ws"].data_ptr(), s["ws"].numel(), stream)
    return s["out"]


def _append_out(s):
    if s["scales"] is None:
        return s["q_out"], s["cache"]
    return s["q_out"], s["cache"].view(torch.float8_e4m3fn), s["scales"]


# ---- plain forms -----------------------------------------------------------------------------
def run(state):
    if own:
        return _run_own(state)
    s, op = state, state["op"]
    if op == "rope":
        c, sn = _angles(s)
        s["out"].copy_(_rotate(s["x"].float().view(s["rows"], s["heads"], s["hd"]), c, sn).view(s["rows"], -1))
        return s["out"]
    if op == "append":
        return _plain_append(s)
    return _plain_step(s) if op == "step" else _plain_prompt(s)


def _angles(s):
    a = s["pos"].double()[s["axis_t"]].t() * s["freq_t"]          # [rows, pairs]
    return torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]


def _rotate(x, c, sn):
    """Pairs (i, i + pairs) of the first 2 * pairs elements of each head turned by their angles."""
    n = c.shape[-1]
    a, b = x[..., :n], x[..., n:2 * n]
    return torch.cat([a * c - b * sn, b * c + a * sn, x[..., 2 * n:]], -1)


def _plain_append(s):
    n, hq, hkv, hd, page = s["rows"], s["hq"], s["hkv"], s["hd"], s["page"]
    c, sn = _angles(s)
    s["q_out"].copy_(_rotate(s["q"].float().view(n, hq, hd), c, sn).view(n, -1))
    k, v = _rotate(s["k"].float().view(n, hkv, hd), c, sn), s["v"].float().view(n, hkv, hd)
    at = s["at"].long()
    pid, off = s["table"][s["seq"].long(), at // page].long(), at % page
    for plane, x in enumerate((k, v)):
        if s["scales"] is None:
            s["cache"][plane][pid, :, off] = x.to(s["cache"].dtype)
        else:
            codes, sc = _quantise(x)
            s["cache"][plane][pid, :, off] = codes.view(torch.uint8)
            s["scales"][plane][pid, :, off] = sc
    return _append_out(s)


def _cached(s, i, a, b):
    """Rows a .. b-1 of sequence i: two fp32 tensors [Hkv, b - a, hd]."""
    page = s["page"]
    p0, p1 = a // page, (b + page - 1) // page
    ids = s["table"][i, p0:p1].long()
    out = []
    for plane in range(2):
        x = s["cache"][plane][ids]
        if s["scales"] is None:
            x = x.float()
        else:
            x = x.view(torch.float8_e4m3fn).float() * s["scales"][plane][ids][..., None]
        x = x.transpose(0, 1).reshape(s["hkv"], -1, s["hd"])
        out.append(x[:, a - p0 * page:b - p0 * page])
    return out


def _visible(s, p, first):
    """The parts of rows 0 .. p that some query of positions first .. p sees: sinks and the window's rows."""
    w = s["window"]
    lo = max(0, first - w + 1) if w else 0
    top = min(s["sinks"], lo)
    return ([(0, top)] if top > 0 else []) + [(lo, p + 1)]


def _plain_step(s):
    hq, hkv, hd = s["hq"], s["hkv"], s["hd"]
    for i, p in enumerate(_step_pos(s)):
        parts = [_cached(s, i, a, b) for a, b in _visible(s, p, p)]
        k, v = (torch.cat([x[j] for x in parts], 1) for j in range(2))
        q = s["q"][i].float().view(hkv, hq // hkv, hd) * hd ** -0.5
        z = q @ k.transpose(1, 2)
        e = torch.exp(z - z.amax(-1, keepdim=True))
        s["out"][i] = ((e @ v) / e.sum(-1, keepdim=True)).view(hq, hd).to(s["out"].dtype)
    return s["out"]


def _plain_prompt(s):
    lens, row0, pos0, _ = _prompts(s)
    hq, hkv, hd, w, dev = s["hq"], s["hkv"], s["hd"], s["window"], s["q"].device
    G, step = hq // hkv, 1024
    for i, (n, r, p0) in enumerate(zip(lens, row0, pos0)):
        for c in range(0, n, step):
            m = min(step, n - c)
            parts = _visible(s, p0 + c + m - 1, p0 + c)
            kv = [_cached(s, i, a, b) for a, b in parts]
            k, v = (torch.cat([x[j] for x in kv], 1) for j in range(2))
            key = torch.cat([torch.arange(a, b, device=dev) for a, b in parts])
            pos = torch.arange(p0 + c, p0 + c + m, device=dev)[:, None]
            seen = key[None] <= pos
            if w:
                seen &= (pos - key[None] < w) | (key[None] < s["sinks"])
            hidden = ~seen.repeat(G, 1)                            # rows of a kv head: [G, m]
            q = s["q"][r + c:r + c + m].float().view(m, hkv, G, hd).permute(1, 2, 0, 3).reshape(hkv, G * m, hd)
            for h in range(hkv):
                z = (q[h] * hd ** -0.5 @ k[h].t()).masked_fill_(hidden, -math.inf)
                e = torch.exp(z - z.amax(-1, keepdim=True))
                o = (e @ v[h]) / e.sum(-1, keepdim=True)
                s["out"][r + c:r + c + m, h * G:(h + 1) * G] = o.view(G, m, hd).transpose(0, 1).to(s["out"].dtype)
    return s["out"]


# ---- necessary work --------------------------------------------------------------------------
def _row_bytes(case):
    """Bytes of one cached row of one head in one plane."""
    return case["hd"] * WIDTH[case["fmt"]] + (4 if case["fmt"] == "e4m3" else 0)


def work(case):
    op, hd = case["op"], case["hd"]
    if op == "rope":
        n = case["rows"] * case["heads"]
        return {"bytes": n * hd * (WIDTH[case["src"]] + WIDTH[case["dst"]]) + 4 * case["axes"] * case["rows"],
                "flops": 3 * n * case["rot"]}
    hq, hkv = case["hq"], case["hkv"]
    if op == "append":
        n = case["rows"]
        return {"bytes": n * ((hq + 2 * hkv) * hd * WIDTH[case["src"]] + 2 * hq * hd + 2 * hkv * _row_bytes(case) +
                              4 * (2 + (case["axes"] if case["axes"] > 1 else 0))),
                "flops": 3 * n * (hq + hkv) * case["rot"]}
    w, sinks = case["window"], case["sinks"]

    def pairs(p0, n):                              # keys seen by the queries at p0 .. p0 + n - 1
        if not w:
            return n * p0 + n * (n + 1) // 2
        total = 0
        for p in range(p0, p0 + n):
            lo = max(0, p - w + 1)
            total += p + 1 - lo + min(sinks, lo)
        return total

    if op == "step":
        lens, pos0 = [1] * case["seqs"], _step_pos(case)
    else:
        lens, _, pos0, _ = _prompts(case)
    keys = sum(pairs(p, n) for n, p in zip(lens, pos0))
    rows = 0
    for n, p in zip(lens, pos0):
        if n:
            lo = max(0, p - w + 1) if w else 0
            rows += p + n - lo + min(sinks, lo)
    return {"bytes": 2 * rows * hkv * _row_bytes(case) + 4 * sum(lens) * hq * hd, "flops": 4 * hd * hq * keys}


# ---- the definitions in 64 bits --------------------------------------------------------------
def _turned(x, pos, freq, axis):
    """[rows, heads, hd] in 64 bits, each pair as a complex number times exp(i angle)."""
    n = len(freq)
    angle = torch.empty(x.shape[0], n, device=x.device, dtype=torch.float64)
    for i in range(n):
        angle[:, i] = pos[axis[i]].to(torch.float64) * freq[i]
    z = torch.complex(x[..., :n].contiguous(), x[..., n:2 * n].contiguous())
    z = z * torch.polar(torch.ones_like(angle), angle)[:, None, :]
    y = x.clone()
    y[..., :n], y[..., n:2 * n] = z.real, z.imag
    return y


def _e4m3(x):
    """Scale 2^E, E the smallest from -126 on with 448 * 2^E >= max |x|, and x / scale on e4m3's grid."""
    a = x.abs().amax(-1)
    sc = torch.exp2(torch.floor(torch.log2(a / 448.0)) - 1)      # at or below the wanted power of two
    for _ in range(3):
        sc = torch.where(448.0 * sc < a, 2 * sc, sc)
    y = x / sc[..., None]
    e = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -1000))).clamp(min=-6)
    step = torch.exp2(e - 3)
    return (torch.round(y / step) * step).clamp(-448.0, 448.0), sc


def _token_rows(s, i, keys, plane):
    """The 64-bit values of sequence i's cached rows `keys`: [len(keys), Hkv, hd]."""
    pid = s["table"][i][torch.div(keys, s["page"], rounding_mode="floor")].long()
    off = torch.remainder(keys, s["page"])
    x = s["cache"][plane, pid, :, off]
    if s["scales"] is None:
        return x.to(torch.float64)
    return x.view(torch.float8_e4m3fn).to(torch.float64) * s["scales"][plane, pid, :, off].to(torch.float64)[..., None]


def exact(case, seed):
    s, op, d = prepare(case, seed), case["op"], torch.float64
    hd = case["hd"]
    if op == "rope":
        x = s["x"].to(d).reshape(case["rows"], case["heads"], hd)
        return _turned(x, s["pos"], s["inv_freq"], s["axis"]).reshape(case["rows"], -1)
    if op == "append":
        n, hkv, page = case["rows"], case["hkv"], case["page"]
        q, k, v = (s[x].to(d).reshape(n, -1, hd) for x in "qkv")
        q_out = _turned(q, s["pos"], s["inv_freq"], s["axis"]).reshape(n, -1)
        k = _turned(k, s["pos"], s["inv_freq"], s["axis"])
        cache = torch.zeros(2, s["n_pages"], hkv, page, hd, device="cuda", dtype=d)
        scales = torch.zeros(2, s["n_pages"], hkv, page, device="cuda", dtype=d)
        place = torch.div(s["at"], page, rounding_mode="floor")
        pid = torch.gather(s["table"][s["seq"].long()], 1, place.long()[:, None])[:, 0].long()
        off = torch.remainder(s["at"], page).long()
        for plane, x in enumerate((k, v)):
            if case["fmt"] == "e4m3":
                x, sc = _e4m3(x)
                for h in range(hkv):
                    scales[plane, pid, h, off] = sc[:, h]
            for h in range(hkv):
                cache[plane, pid, h, off] = x[:, h]
        return (q_out, cache, scales) if case["fmt"] == "e4m3" else (q_out, cache)
    hq, hkv, w, sinks = case["hq"], case["hkv"], case["window"], case["sinks"]
    out = torch.zeros(s["q"].shape[0], hq, hd, device="cuda", dtype=d)
    if op == "step":
        todo = [(i, i, 1, p) for i, p in enumerate(_step_pos(case))]
    else:
        lens, row0, pos0, _ = _prompts(case)
        todo = [(i, r + c, min(512, n - c), p + c) for i, (n, r, p) in enumerate(zip(lens, row0, pos0))
                for c in range(0, n, 512)]
    for i, r, m, p in todo:                        # m queries of sequence i from row r, position p on
        keys = torch.arange(p + m, device="cuda")
        if w:
            keys = keys[(keys < sinks) | (keys > p - w)]
        back = torch.arange(p, p + m, device="cuda")[:, None] - keys[None, :]
        bias = torch.zeros(m, len(keys), device="cuda", dtype=d)
        bias[back < 0] = -math.inf
        if w:
            bias[(back >= w) & (keys[None, :] >= sinks)] = -math.inf
        k, v = _token_rows(s, i, keys, 0), _token_rows(s, i, keys, 1)
        for j in range(hq):
            h = j * hkv // hq
            z = s["q"][r:r + m, j * hd:(j + 1) * hd].to(d) @ k[:, h].t() / math.sqrt(hd) + bias
            out[r:r + m, j] = torch.softmax(z, 1) @ v[:, h]
    return out
