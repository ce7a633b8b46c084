"""Refusals of the stream-ordered operators over a shared prefix: every bad argument is reported
before any device work, so these run without a GPU (pointers are never followed)."""
import ctypes as C

import numpy as np
import pytest

from prefill_only_decision_gb300 import build


@pytest.fixture(scope="module")
def B():
    build.build()
    from prefill_only_decision_gb300 import binding
    binding.lib()
    return binding


P = 1 << 20      # a 16-byte aligned stand-in for a device pointer
ARG, UNSUP = 1, 7


def refused(B, code, f, **kw):
    with pytest.raises(B.S1Error) as e:
        f(**kw)
    assert e.value.code == code, e.value


KV = dict(k=P, v=P, dtype=2, k_stride=512, v_stride=512, n_rows=4, Hkv=4, hd=128, codes=P, scales=P, cap=16, pos0=0)


@pytest.mark.parametrize("bad,code", [
    (dict(dtype=3), ARG), (dict(dtype=-1), ARG), (dict(n_rows=-1), ARG), (dict(n_rows=17), ARG),
    (dict(pos0=13), ARG), (dict(pos0=-1), ARG), (dict(pos0=2**31 - 2, n_rows=4), ARG), (dict(Hkv=0), ARG),
    (dict(hd=96), UNSUP), (dict(hd=256), UNSUP), (dict(k_stride=511), ARG), (dict(v_stride=-512), ARG),
    (dict(k=0), ARG), (dict(v=0), ARG), (dict(codes=0), ARG), (dict(scales=0), ARG), (dict(k=P + 1), ARG),
    (dict(codes=P + 8), ARG), (dict(scales=P + 2), ARG), (dict(dtype=0, v=P + 2), ARG), (dict(Hkv=70000), UNSUP),
])
def test_kv_refusals(B, bad, code):
    refused(B, code, B.op_kv_quant_async, **{**KV, **bad})
    refused(B, code, B.op_kv_dequant_async, **{**KV, **bad})


def test_kv_nothing_to_do(B):
    B.op_kv_quant_async(**{**KV, "n_rows": 0, "k": 0, "codes": 0})
    B.op_kv_dequant_async(**{**KV, "n_rows": 0, "pos0": 16})


AT = dict(q=P, q_stride=2048, k_new=P, v_new=P, kv_stride=512, row0=[0, 8], lens=[8, 3], kv=P, scales=0, kv_format=0,
          P=100, cap=128, Hq=16, Hkv=4, hd=128, sm_scale=0.1, out=P, workspace=P, workspace_bytes=1 << 40)


@pytest.mark.parametrize("bad,code", [
    (dict(Hq=15), ARG), (dict(Hq=0), ARG), (dict(Hkv=0), ARG), (dict(hd=80), UNSUP), (dict(P=-1), ARG),
    (dict(P=129), ARG), (dict(Hq=129, Hkv=1, q_stride=129 * 128), UNSUP), (dict(kv_format=2), ARG),
    (dict(row0=[0, 7]), ARG), (dict(row0=[8, 0]), ARG), (dict(row0=[-1, 8]), ARG), (dict(lens=[-1, 3]), ARG),
    (dict(row0=[0, 2**31 - 3]), ARG), (dict(k_new=0), ARG), (dict(v_new=0), ARG), (dict(q_stride=2047), ARG),
    (dict(q_stride=2052), ARG), (dict(kv_stride=504), ARG), (dict(kv_stride=516), ARG), (dict(q=0), ARG),
    (dict(out=0), ARG), (dict(kv=0), ARG), (dict(kv_format=1), ARG), (dict(q=P + 8), ARG), (dict(k_new=P + 2), ARG),
    (dict(out=P + 4), ARG), (dict(kv=P + 8), ARG), (dict(kv_format=1, scales=P + 1), ARG), (dict(workspace=P + 8), ARG),
    (dict(sm_scale=0.0), ARG), (dict(sm_scale=-1.0), ARG), (dict(sm_scale=float("nan")), ARG),
    (dict(sm_scale=float("inf")), ARG),
])
def test_attention_refusals(B, bad, code):
    refused(B, code, B.op_attention_shared_async, **{**AT, **bad})


def test_attention_workspace_is_required(B):
    """A size that needs a workspace is refused without one and with one byte too few."""
    big = {**AT, "P": 100000, "cap": 100000}
    need = B.op_attention_shared_workspace(big["lens"], big["P"], 16, 4, 128)
    if need:
        refused(B, ARG, B.op_attention_shared_async, **{**big, "workspace": 0})
        refused(B, ARG, B.op_attention_shared_async, **{**big, "workspace_bytes": need - 1})
    refused(B, ARG, B.op_attention_shared_workspace, lens=[1], P=-1, Hq=16, Hkv=4, hd=128)
    refused(B, ARG, B.op_attention_shared_workspace, lens=[-1], P=1, Hq=16, Hkv=4, hd=128)


def test_attention_nothing_to_do(B):
    B.op_attention_shared_async(**{**AT, "row0": [], "lens": []})
    B.op_attention_shared_async(**{**AT, "lens": [0, 0], "q": 0, "out": 0})


LA = dict(q=P, k=P, v=P, dtype=2, q_stride=1024, k_stride=1024, v_stride=1024, log_decay=P, H=8, dk=128, dv=128,
          scale=0.1, S_in=0, s_in_stride=0, S_out=0, out=P)
PER = 8 * 128 * 128
LIN_BAD = [
    (dict(dtype=0), ARG), (dict(dtype=9), ARG), (dict(H=0), ARG), (dict(dk=96), UNSUP), (dict(dv=256), UNSUP),
    (dict(q_stride=1016), ARG), (dict(k_stride=1028), ARG), (dict(v_stride=-1024), ARG), (dict(q=0), ARG),
    (dict(k=0), ARG), (dict(v=0), ARG), (dict(log_decay=0), ARG), (dict(out=0), ARG), (dict(q=P + 2), ARG),
    (dict(out=P + 8), ARG), (dict(S_in=P + 4), ARG), (dict(S_out=P + 4), ARG), (dict(log_decay=P + 2), ARG),
    (dict(S_in=P, s_in_stride=5), ARG), (dict(S_in=P, s_in_stride=-PER), ARG),
    (dict(S_in=P, s_in_stride=0, S_out=P), ARG),                    # one shared state advanced in place
    (dict(S_in=P, s_in_stride=PER, S_out=P + 4 * PER), ARG),        # states shifted by one
    (dict(S_in=P + 16, s_in_stride=0, S_out=P), ARG),
    (dict(H=5000, q_stride=5000 * 128, k_stride=5000 * 128, v_stride=5000 * 128), UNSUP),
]


@pytest.mark.parametrize("bad,code", LIN_BAD)
def test_linattn_refusals(B, bad, code):
    kw = {**LA, **bad}
    refused(B, code, B.op_linattn_step_async, n=3, **kw)
    refused(B, code, B.op_linattn_async, row0=[0, 5, 9], lens=[5, 4, 1], workspace=P, workspace_bytes=1 << 40, **kw)


@pytest.mark.parametrize("bad", [dict(row0=[0, 4, 9]), dict(row0=[0, 5, 8]), dict(lens=[5, -4, 1]),
                                 dict(row0=[0, 5, 2**31 - 1]), dict(workspace=P + 8)])
def test_linattn_sequence_refusals(B, bad):
    kw = dict(row0=[0, 5, 9], lens=[5, 4, 1], workspace=P, workspace_bytes=1 << 40, **LA)
    refused(B, ARG, B.op_linattn_async, **{**kw, **bad})


def test_linattn_workspace(B):
    kw = dict(row0=[0], lens=[70001], workspace=P, **LA)
    need = B.op_linattn_workspace([70001], 8, 128, 128)
    if need:
        refused(B, ARG, B.op_linattn_async, **{**kw, "workspace": 0, "workspace_bytes": need})
        refused(B, ARG, B.op_linattn_async, **{**kw, "workspace_bytes": need - 1})
    refused(B, ARG, B.op_linattn_workspace, lens=[-1], H=8, dk=128, dv=128)
    refused(B, UNSUP, B.op_linattn_workspace, lens=[1], H=8, dk=128, dv=100)


def test_linattn_nothing_to_do(B):
    B.op_linattn_async(row0=[], lens=[], workspace=0, workspace_bytes=0, **LA)
    B.op_linattn_step_async(n=0, **LA)
    refused(B, ARG, B.op_linattn_step_async, n=-1, **LA)


def test_mismatched_sequence_arrays(B):
    with pytest.raises(ValueError):
        B.op_attention_shared_async(**{**AT, "row0": [0]})


def test_null_outputs_of_the_sizing_calls(B):
    ln = np.array([4], np.int32)
    assert B.lib().s1_op_linattn_workspace(1, ln.ctypes.data, 8, 128, 128, None) == ARG
    assert B.lib().s1_op_attention_shared_workspace(1, ln.ctypes.data, 4, 8, 2, 128, None) == ARG
    out = C.c_int64()
    assert B.lib().s1_op_attention_shared_workspace(1, None, 4, 8, 2, 128, C.byref(out)) == ARG


@pytest.mark.parametrize("bad", [np.array([2 ** 32, 2 ** 32 + 8]), np.array([0, 2 ** 31]), [0, 2 ** 40], [0.0, 8.5],
                                 np.array([0, -2 ** 31 - 1]), [[0, 8]], np.array([0, 2 ** 63], np.uint64)])
def test_sequence_arrays_are_not_wrapped(B, bad):
    """Rows and lengths that 32 bits cannot hold, fractions and tables are refused; they would become other rows."""
    with pytest.raises(ValueError):
        B.op_attention_shared_async(**{**AT, "row0": bad})
    kw = dict(workspace=P, workspace_bytes=1 << 40, **LA)
    with pytest.raises(ValueError):
        B.op_linattn_async(row0=bad, lens=[8, 3], **kw)
    with pytest.raises(ValueError):
        B.op_linattn_async(row0=[0, 8], lens=bad, **kw)
    with pytest.raises(ValueError):
        B.op_linattn_workspace(bad, 8, 128, 128)
    with pytest.raises(ValueError):
        B.op_attention_shared_workspace(bad, 100, 16, 4, 128)


@pytest.mark.parametrize("lens", [[5, 0, 7], np.array([5, 0, 7]), np.array([5, 9, 0, 9, 7])[::2], (5, 0, 7),
                                  np.array([5, 0, 7], np.uint8)])
def test_sequence_arrays_of_other_types(B, lens):
    want = B.op_linattn_workspace(np.array([5, 0, 7], np.int32), 8, 128, 128)
    assert B.op_linattn_workspace(lens, 8, 128, 128) == want
    assert B.op_linattn_workspace([], 8, 128, 128) == 0


BIG = 2 ** 32


def test_sizes_are_not_cut(B):
    """A size beyond 32 bits is refused; cut to its low half it would be another one."""
    for name in ("n_rows", "cap", "pos0", "Hkv", "hd"):
        for f in (B.op_kv_quant_async, B.op_kv_dequant_async):
            with pytest.raises(ValueError):
                f(**{**KV, name: KV[name] + BIG})
    for name in ("P", "cap", "Hq", "Hkv", "hd"):
        with pytest.raises(ValueError):
            B.op_attention_shared_async(**{**AT, name: AT[name] + BIG})
    for name in ("H", "dk", "dv"):
        with pytest.raises(ValueError):
            B.op_linattn_async(row0=[0], lens=[5], workspace=P, workspace_bytes=1 << 40, **{**LA, name: LA[name] + BIG})
        with pytest.raises(ValueError):
            B.op_linattn_step_async(n=3, **{**LA, name: LA[name] - 2 * BIG})
    with pytest.raises(ValueError):
        B.op_linattn_step_async(n=3 + BIG, **LA)
    with pytest.raises(ValueError):
        B.op_attention_shared_workspace([4], P=100 + BIG, Hq=16, Hkv=4, hd=128)
    with pytest.raises(ValueError):
        B.op_linattn_workspace([4], 8 + BIG, 128, 128)
