"""Refusals of the stream-ordered operators around a paged cache: every bad argument is reported before
any device work, so these run without a GPU (pointers are never followed)."""
import ctypes as C

import numpy as np
import pytest

from test_shared_ops_args import ARG, BIG, P, UNSUP, B, refused  # noqa: F401  (B: the fixture)

INF, NAN = float("inf"), float("nan")


def rope(B, n_pairs=64, n_axes=3, freq=None, axis=None):
    w = np.full(n_pairs, 0.5) if freq is None else np.full(n_pairs, freq)
    return B.Rope(w, np.arange(n_pairs) % 3 if axis is None else np.full(n_pairs, axis), n_axes)


ROPE = dict(x=P, dtype=2, x_stride=512, n_rows=4, H=4, hd=128, pos=P, pos_stride=4, out=2 * P, out_dtype=2,
            out_stride=512)


@pytest.mark.parametrize("bad,code", [
    (dict(dtype=3), ARG), (dict(out_dtype=-1), ARG), (dict(out_dtype=1), ARG), (dict(out_dtype=0), ARG),
    (dict(dtype=1), ARG), (dict(n_rows=-1), ARG), (dict(H=0), ARG), (dict(hd=96), UNSUP), (dict(hd=256), UNSUP),
    (dict(H=70000, x_stride=70000 * 128, out_stride=70000 * 128), UNSUP), (dict(x_stride=511), ARG),
    (dict(out_stride=-512), ARG), (dict(pos_stride=3), ARG), (dict(x=0), ARG), (dict(pos=0), ARG), (dict(out=0), ARG),
    (dict(x=P + 1), ARG), (dict(out=2 * P + 1), ARG), (dict(pos=P + 2), ARG), (dict(dtype=0, x=P + 2, out_dtype=2), ARG),
    (dict(out=P, out_stride=520), ARG), (dict(dtype=0, out=P), ARG)])
def test_rope_refusals(B, bad, code):
    refused(B, code, B.op_rope_async, rope=rope(B), **{**ROPE, **bad})


@pytest.mark.parametrize("spec,code", [
    (dict(n_pairs=0), ARG), (dict(n_pairs=12), ARG), (dict(n_pairs=72), ARG), (dict(n_axes=0), ARG), (dict(n_axes=5), ARG),
    (dict(n_axes=2), ARG), (dict(axis=3), ARG), (dict(freq=NAN), ARG), (dict(freq=-INF), ARG)])
def test_rope_specs(B, spec, code):
    refused(B, code, B.op_rope_async, rope=rope(B, **spec), **ROPE)
    if spec.get("n_pairs") != 0:
        refused(B, code, B.op_kv_append_async, **append(B, rope=rope(B, **spec)))


def test_rope_spec_itself(B):
    refused(B, ARG, B.op_rope_async, rope=None, **ROPE)
    for bad in (dict(inv_freq=[1.0] * 8, axis=[0] * 7), dict(inv_freq=[[1.0] * 8]), dict(inv_freq=[1.0] * 8, axis=[256] * 8),
                dict(inv_freq=[1.0] * 8, axis=[-1] * 8), dict(inv_freq=[1.0] * 8, axis=[0.5] * 8)):
        with pytest.raises(ValueError):
            B.Rope(**bad)
    r = B.Rope([1.0] * 8)
    r.inv_freq = None
    refused(B, ARG, B.op_rope_async, rope=r, **ROPE)


PG = dict(data=P, scales=0, format=0, n_pages=10, page_rows=16, Hkv=4, hd=128, table=P, n_seq=5, cols=8)


def pages(B, **kw):
    return B.KvPages(**{**PG, **kw})


BAD_PAGES = [
    (dict(data=0), ARG), (dict(data=P + 8), ARG), (dict(format=3), ARG), (dict(format=-1), ARG), (dict(format=1), ARG),
    (dict(scales=P), ARG), (dict(format=1, scales=P + 2), ARG), (dict(n_pages=0), ARG), (dict(page_rows=8), UNSUP),
    (dict(page_rows=48), UNSUP), (dict(page_rows=256), UNSUP), (dict(page_rows=0), UNSUP), (dict(Hkv=0), ARG),
    (dict(Hkv=5000), UNSUP), (dict(hd=96), UNSUP), (dict(table=0), ARG), (dict(table=P + 2), ARG), (dict(n_seq=-1), ARG),
    (dict(cols=-1), ARG), (dict(table_stride=7), ARG), (dict(cols=2 ** 27, table_stride=2 ** 27), UNSUP)]


def append(B, **kw):
    kw.setdefault("pages", pages(B))
    kw.setdefault("rope", rope(B))
    return {**dict(q=P, k=P, v=P, dtype=2, q_stride=2048, k_stride=512, v_stride=512, n_rows=4, Hq=16, pos=P, pos_stride=4,
                   seq=P, at=P, q_out=P, q_dtype=2), **kw}


def step(B, **kw):
    kw.setdefault("pages", pages(B))
    return {**dict(q=P, q_dtype=2, q_stride=2048, n=4, Hq=16, pos=P, window=0, sinks=0, sm_scale=0.1, out=P, workspace=P,
                   workspace_bytes=1 << 40), **kw}


def prompt(B, **kw):
    kw.setdefault("pages", pages(B))
    return {**dict(q=P, q_dtype=2, q_stride=2048, row0=[0, 8], lens=[8, 3], pos0=[0, 7], Hq=16, window=0, sinks=0,
                   sm_scale=0.1, out=P, workspace=P, workspace_bytes=1 << 40), **kw}


@pytest.mark.parametrize("bad,code", BAD_PAGES)
def test_pages_refusals(B, bad, code):
    pg = pages(B, **bad)
    refused(B, code, B.op_kv_append_async, **append(B, pages=pg))
    refused(B, code, B.op_attention_paged_step_async, **step(B, pages=pg))
    refused(B, code, B.op_attention_paged_async, **prompt(B, pages=pg))


def test_pages_null(B):
    refused(B, ARG, B.op_kv_append_async, **{**append(B), "pages": None})
    refused(B, ARG, B.op_attention_paged_step_async, **{**step(B), "pages": None})
    refused(B, ARG, B.op_attention_paged_async, **{**prompt(B), "pages": None})


@pytest.mark.parametrize("bad,code", [
    (dict(dtype=3), ARG), (dict(q_dtype=0), ARG), (dict(n_rows=-1), ARG), (dict(Hq=-1), ARG), (dict(q_stride=2047), ARG),
    (dict(k_stride=511), ARG), (dict(v_stride=-512), ARG), (dict(pos_stride=3), ARG), (dict(seq=0, n_rows=6, pos_stride=6), ARG),
    (dict(q=0), ARG), (dict(Hq=0), ARG), (dict(k=0), ARG), (dict(v=0), ARG), (dict(at=0), ARG), (dict(q_out=0), ARG),
    (dict(k=P + 1), ARG), (dict(dtype=0, v=P + 2), ARG), (dict(at=P + 2), ARG), (dict(seq=P + 1), ARG),
    (dict(pos=P + 2), ARG), (dict(q_out=P + 1), ARG), (dict(Hq=40000, q_stride=40000 * 128), UNSUP)])
def test_append_refusals(B, bad, code):
    refused(B, code, B.op_kv_append_async, **append(B, **bad))


HEADS = [(dict(Hq=15), ARG), (dict(Hq=0), ARG), (dict(Hq=4 * 129, q_stride=4 * 129 * 128), UNSUP)]
ATTN = HEADS + [
    (dict(q_dtype=0), ARG), (dict(q_dtype=1), ARG), (dict(q_stride=2040), ARG), (dict(q_stride=2052), ARG),
    (dict(window=-1), ARG), (dict(sinks=-1), ARG), (dict(sm_scale=0.0), ARG), (dict(sm_scale=-1.0), ARG),
    (dict(sm_scale=NAN), ARG), (dict(sm_scale=INF), ARG), (dict(q=0), ARG), (dict(out=0), ARG), (dict(q=P + 8), ARG),
    (dict(out=P + 4), ARG), (dict(workspace=P + 8), ARG)]


@pytest.mark.parametrize("bad,code", ATTN + [(dict(n=-1), ARG), (dict(n=6), ARG), (dict(pos=0), ARG), (dict(pos=P + 2), ARG)])
def test_step_refusals(B, bad, code):
    refused(B, code, B.op_attention_paged_step_async, **step(B, **bad))


@pytest.mark.parametrize("bad,code", ATTN + [
    (dict(row0=[0, 7]), ARG), (dict(row0=[8, 0]), ARG), (dict(lens=[-1, 3]), ARG), (dict(pos0=[0, -1]), ARG),
    (dict(pos0=[0, 126]), ARG), (dict(row0=[0, 2 ** 31 - 3]), ARG),
    (dict(row0=range(6), lens=[1] * 6, pos0=[0] * 6), ARG)])
def test_prompt_refusals(B, bad, code):
    refused(B, code, B.op_attention_paged_async, **prompt(B, **bad))


def test_queries_have_the_pages_type(B):
    bf = pages(B, format=2)
    refused(B, ARG, B.op_attention_paged_step_async, **step(B, pages=bf))
    refused(B, ARG, B.op_attention_paged_async, **prompt(B, pages=bf))


def test_workspaces_are_required(B):
    need = B.op_attention_paged_step_workspace(4, 16, 4, 128)
    if need:
        refused(B, ARG, B.op_attention_paged_step_async, **step(B, workspace=0))
        refused(B, ARG, B.op_attention_paged_step_async, **step(B, workspace_bytes=need - 1))
    kw = dict(pages=pages(B, cols=10000), lens=[8, 3], pos0=[0, 100000])
    need = B.op_attention_paged_workspace(kw["lens"], kw["pos0"], 16, 4, 128, 0, 0)
    if need:
        refused(B, ARG, B.op_attention_paged_async, **prompt(B, **kw, workspace=0))
        refused(B, ARG, B.op_attention_paged_async, **prompt(B, **kw, workspace_bytes=need - 1))


@pytest.mark.parametrize("bad,code", [(dict(n=-1), ARG), (dict(Hq=15), ARG), (dict(Hkv=0), ARG), (dict(hd=96), UNSUP)])
def test_step_workspace_refusals(B, bad, code):
    refused(B, code, B.op_attention_paged_step_workspace, **{**dict(n=4, Hq=16, Hkv=4, hd=128), **bad})


@pytest.mark.parametrize("bad,code", [(dict(lens=[-1]), ARG), (dict(pos0=[-1]), ARG), (dict(pos0=[2 ** 31 - 2]), ARG),
                                      (dict(Hq=15), ARG), (dict(hd=80), UNSUP), (dict(window=-1), ARG), (dict(sinks=-1), ARG)])
def test_prompt_workspace_refusals(B, bad, code):
    refused(B, code, B.op_attention_paged_workspace,
            **{**dict(lens=[4], pos0=[9], Hq=16, Hkv=4, hd=128, window=0, sinks=0), **bad})


def test_calls_too_large(B):
    """Sizes whose numbers of tiles or items leave 31 bits."""
    big = pages(B, n_seq=4096, cols=2 ** 23, Hkv=64, page_rows=128)
    refused(B, UNSUP, B.op_attention_paged_step_async, **step(B, pages=big, n=4096, Hq=64, q_stride=64 * 128))
    refused(B, UNSUP, B.op_attention_paged_async,
            **prompt(B, pages=big, row0=[0], lens=[2 ** 29], pos0=[0], Hq=64, q_stride=64 * 128))
    refused(B, UNSUP, B.op_attention_paged_workspace, lens=[2 ** 30], pos0=[0], Hq=64, Hkv=64, hd=128, window=0, sinks=0)
    assert B.op_attention_paged_workspace([4], [2 ** 30], 4, 4, 128, 0, 0) > 0      # more than 64 parts


def test_null_outputs_of_the_sizing_calls(B):
    one = np.array([4], np.int32)
    out = C.c_int64()
    L = B.lib()
    assert L.s1_op_attention_paged_step_workspace(1, 8, 2, 128, None) == ARG
    assert L.s1_op_attention_paged_workspace(1, one.ctypes.data, one.ctypes.data, 8, 2, 128, 0, 0, None) == ARG
    assert L.s1_op_attention_paged_workspace(1, None, one.ctypes.data, 8, 2, 128, 0, 0, C.byref(out)) == ARG
    assert L.s1_op_attention_paged_workspace(1, one.ctypes.data, None, 8, 2, 128, 0, 0, C.byref(out)) == ARG


def test_nothing_to_do(B):
    B.op_rope_async(rope=rope(B), **{**ROPE, "n_rows": 0, "x": 0, "out": 0, "pos": 0})
    B.op_kv_append_async(**append(B, n_rows=0, k=0, v=0, q=0, q_out=0, at=0))
    B.op_attention_paged_step_async(**step(B, n=0, q=0, out=0, pos=0))
    B.op_attention_paged_async(**prompt(B, row0=[], lens=[], pos0=[], q=0))
    B.op_attention_paged_async(**prompt(B, lens=[0, 0], q=0, out=0))


def test_sizes_are_not_cut(B):
    for name in ("n_rows", "H", "hd"):
        with pytest.raises(ValueError):
            B.op_rope_async(rope=rope(B), **{**ROPE, name: ROPE[name] + BIG})
    for name in ("format", "n_pages", "page_rows", "Hkv", "hd", "n_seq", "cols"):
        with pytest.raises(ValueError):
            pages(B, **{name: PG[name] + BIG})
    for name in ("n_rows", "Hq"):
        with pytest.raises(ValueError):
            kw = append(B)
            B.op_kv_append_async(**{**kw, name: kw[name] + BIG})
    for name in ("Hq", "window", "sinks"):
        for f, kw in ((B.op_attention_paged_step_async, step(B)), (B.op_attention_paged_async, prompt(B))):
            with pytest.raises(ValueError):
                f(**{**kw, name: kw[name] + BIG})
    with pytest.raises(ValueError):
        B.op_attention_paged_step_async(**step(B, n=4 + BIG))
    for bad in (np.array([0, 2 ** 32]), [0.0, 7.5], [[0, 7]], [0]):
        with pytest.raises(ValueError):
            B.op_attention_paged_async(**prompt(B, pos0=bad))
        with pytest.raises(ValueError):
            B.op_attention_paged_workspace([8, 3], bad, 16, 4, 128, 0, 0)
