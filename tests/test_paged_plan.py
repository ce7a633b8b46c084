"""Plans of prompts over pages, made on the host: batches with empty sequences, alone and behind others."""
import subprocess
import sys

import numpy as np
import pytest

from prefill_only_decision_gb300 import build

HEADS = dict(Hq=16, Hkv=4, hd=128, window=0, sinks=0)


@pytest.fixture(scope="module")
def B():
    build.build()
    from prefill_only_decision_gb300 import binding
    binding.lib()
    return binding


# A launch takes up to 1024 sequences that are not empty; what comes behind them is a plan of its own.
EMPTY = [([0], [9]), ([0] * 3, [0, 7, 2000]), ([1] * 1024 + [0], [0] * 1025), ([0] * 5 + [3] * 1024 + [0] * 2000, [0] * 3029)]


@pytest.mark.parametrize("lens,pos0", EMPTY)
def test_empty_sequences_are_sized(B, lens, pos0):
    """In a process of its own, so that a plan that divides by their number of tiles fails this test alone."""
    code = ("from prefill_only_decision_gb300 import binding as B\n"
            f"print(B.op_attention_paged_workspace({lens}, {pos0}, 16, 4, 128, 0, 0))")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=build.ROOT)
    assert r.returncode == 0, (r.returncode, r.stderr)
    live = [(n, p) for n, p in zip(lens, pos0) if n]
    want = B.op_attention_paged_workspace(*zip(*live), **HEADS) if live else 0
    assert int(r.stdout) == want


def test_empty_sequences_change_nothing(B):
    """The workspace is that of the sequences that have rows, wherever empty ones stand between them."""
    g = np.random.default_rng(0)
    for _ in range(20):
        lens = g.integers(0, 3, 40) * g.integers(1, 400, 40)
        pos0 = g.integers(0, 60000, 40)
        keep = lens > 0
        assert (B.op_attention_paged_workspace(lens, pos0, **HEADS) ==
                B.op_attention_paged_workspace(lens[keep], pos0[keep], **HEADS))
