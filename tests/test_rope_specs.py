"""Frequencies that the rotary operators take: those whose turns they hold to 2^-64."""
import numpy as np
import pytest

from test_paged_ops_args import ROPE, append, rope
from test_shared_ops_args import UNSUP, B, refused  # noqa: F401  (B: the fixture)


@pytest.mark.parametrize("freq", [np.nextafter(2.0 ** 40, np.inf), -2.0 ** 41, 2.0 ** 53 + 2, 1e300])
def test_frequencies_past_what_is_held(B, freq):  # noqa: F811
    spec = rope(B, freq=freq)
    refused(B, UNSUP, B.op_rope_async, rope=spec, **ROPE)
    refused(B, UNSUP, B.op_kv_append_async, **append(B, rope=spec))


@pytest.mark.parametrize("freq", [2.0 ** 40, -2.0 ** 40, 0.0, 5e-324])
def test_frequencies_that_are_taken(B, freq):  # noqa: F811
    B.op_rope_async(rope=rope(B, freq=freq), **{**ROPE, "n_rows": 0})
