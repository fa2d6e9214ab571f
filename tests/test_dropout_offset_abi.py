"""offset_dev inside an output (no GPU): the kernels read it while they write the
outputs, so the calls refuse it before any HIP call."""

import pytest

from test_training_abi import FAKE, FORMS, INVALID, call, drop


@pytest.mark.parametrize("form", FORMS)
def test_offset_in_an_output_is_refused(form):
    out = FAKE + (1 << 36)  # rank r's output lies at out + r 2^24: 1024 bfloat16 values, or 256 of a shard
    for at in (out, out + 504, out + 3 * (1 << 24)):
        st, msg = call(form, params=drop(0.1, at))
        assert st == INVALID and "offset_dev" in msg, (form, at)
