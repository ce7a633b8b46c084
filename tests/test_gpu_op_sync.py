"""s1_op_sync: what it reports of the operators' bounded waits, for each kernel's word. A wait that gives up writes the time
into its kernel's word on the device; the words are written here instead."""
import ctypes as C
import threading

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

WORDS = ["attention_shared", "linattn", "attention_step", "attention_paged"]


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from prefill_only_decision_gb300 import binding
    binding.lib()
    return binding


def word(B, name):
    """The word of a kernel as a tensor."""
    f = getattr(B.lib(), f"_ZN2s1{len(name) + 13}{name}_gave_up_wordEPPm")
    f.restype, f.argtypes = C.c_int, [C.POINTER(C.c_void_p)]
    at = C.c_void_p()
    assert f(C.byref(at)) == 0 and at.value

    class View:
        __cuda_array_interface__ = dict(shape=(1,), typestr="<i8", data=(at.value, False), version=2)

    return torch.as_tensor(View(), device="cuda")


@pytest.mark.parametrize("name", WORDS)
def test_each_wait_that_gave_up_is_told_of_once(B, name):
    st = torch.cuda.current_stream().cuda_stream
    other = torch.cuda.Stream()
    B.op_sync(st)
    w = word(B, name)
    for stream in (st, other.cuda_stream):
        w += 1000
        torch.cuda.synchronize()
        with pytest.raises(B.S1Error) as e:
            B.op_sync(stream)
        assert e.value.code == B.S1_ERR_DEVICE_TIMEOUT
        B.op_sync(st)
        B.op_sync(other.cuda_stream)


def test_callers_at_once(B):
    """Four threads on streams of their own: one of them is told, and only of what there was."""
    B.op_sync(torch.cuda.current_stream().cuda_stream)
    streams = [torch.cuda.Stream() for _ in range(4)]
    told = []

    def sync(s, rounds):
        for _ in range(rounds):
            try:
                B.op_sync(s.cuda_stream)
            except B.S1Error as e:
                told.append(e.code)

    def together(rounds):
        t = [threading.Thread(target=sync, args=(s, rounds)) for s in streams]
        [x.start() for x in t]
        [x.join() for x in t]

    together(100)
    assert not told
    word(B, "attention_step").add_(1000)
    torch.cuda.synchronize()
    together(20)
    assert told == [B.S1_ERR_DEVICE_TIMEOUT]
